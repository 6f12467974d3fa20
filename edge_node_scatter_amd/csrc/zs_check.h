// Checks of arguments shared by the C ABI's translation units (host code only).
#pragma once

#include <hip/hip_runtime.h>

#include "zs_block.h"

namespace zs {
namespace check {

// Largest extent of a strided view in elements; byte extents and every index
// the kernels form then stay inside int64.
constexpr int64_t kMaxExtent = int64_t(1) << 60;

// Elements that `rows` rows of `width` at `stride` span, -1 if above the limit.
inline int64_t extent(int64_t rows, int64_t stride, int64_t width) {
    if (rows <= 0) return 0;
    int64_t e = 0;
    if (__builtin_mul_overflow(rows - 1, stride, &e) || __builtin_add_overflow(e, width, &e) ||
        e > kMaxExtent)
        return -1;
    return e;
}

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};
inline Range span(const void* p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, p ? lo + uintptr_t(bytes) : lo};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// Whether some output overlaps an input or another output.
inline bool aliased(const Range* outs, int n_outs, const Range* ins, int n_ins) {
    for (int i = 0; i < n_outs; ++i) {
        for (int j = i + 1; j < n_outs; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < n_ins; ++j)
            if (overlap(outs[i], ins[j])) return true;
    }
    return false;
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? ZS_OK : ZS_ERR_HIP; }
inline bool dtype_ok(int d) { return d == ZS_F32 || d == ZS_BF16; }
inline int64_t size_of(int d) { return d == ZS_F32 ? 4 : 2; }

}  // namespace check
}  // namespace zs
