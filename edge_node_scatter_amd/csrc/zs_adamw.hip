// The AdamW step over many tensors, with states in 32 or in 8 bits, gfx950.
//
// One launch takes up to kMaxTensors tensors, described in its kernel
// arguments (no table is copied to the device).  A workgroup of four
// wavefronts takes a run of 256-element blocks of one tensor; in the 8-bit
// form a wavefront holds one block, four elements a lane, so that a block's
// largest magnitude is a reduction over the wavefront.
// Every operation is rounded to fp32 in the order the header gives (the
// sources are compiled without fused multiply-adds), so results do not depend
// on the split.
//
// Bound by memory: 28 bytes an element in fp32 (parameter and moments read and
// written, gradient read), the same with a bf16 gradient and copy; 16 with 8-bit
// moments.  Measured on MI355X: 120 million parameters in 28 tensors, bf16 gradients
// and copies, 644 us, 5.2 TB/s, a copy's rate; 24 million with 8-bit moments 81 to
// 91 us, 4.2 to 4.7 TB/s (some 60 instructions an element for codes, hash and
// rounding beside the memory); 24 small tensors 4.8 us, one launch.
#include "zs_block_internal.h"
#include "zs_tile.h"

namespace zs {

namespace {

constexpr int kMaxTensors = 64;
constexpr int kBlock = ZS_ADAMW_BLOCK;

struct Slice {
    float* p;
    const void* g;
    uint16_t* copy;
    int64_t n, offset;
    uint32_t first;    // first work item of the tensor
    uint32_t flags;    // 1: bf16 gradient, 2: all arrays aligned for 4-element accesses
};

struct Slices {
    Slice s[kMaxTensors];
    int count;
    int blocks_per_item;   // 256-element blocks of a work item
};

__device__ inline int find_slice(const Slices& t, uint32_t item) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.s[mid].first <= item) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ inline float bf16_value(uint16_t b) { return __builtin_bit_cast(float, uint32_t(b) << 16); }
__device__ inline uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, __bf16(f)); }

// Up to four elements i .. i + 3 of a slice; `count` of them exist.
__device__ inline f32x4 load_param4(const float* p, bool wide, int count) {
    if (wide && count >= 4) return *reinterpret_cast<const f32x4*>(p);
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (q < count) v[q] = p[q];
    return v;
}
__device__ inline f32x4 load_grad4(const Slice& s, int64_t i, bool wide, int count) {
    if (!(s.flags & 1)) return load_param4(static_cast<const float*>(s.g) + i, wide, count);
    const uint16_t* p = static_cast<const uint16_t*>(s.g) + i;
    f32x4 v = {0, 0, 0, 0};
    if (wide && count >= 4) {
        const u32x2 raw = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            v[2 * q] = __builtin_bit_cast(float, raw[q] << 16);
            v[2 * q + 1] = __builtin_bit_cast(float, raw[q] & 0xffff0000u);
        }
        return v;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (q < count) v[q] = bf16_value(p[q]);
    return v;
}
__device__ inline void store_param4(const Slice& s, int64_t i, bool wide, int count, f32x4 v) {
    if (wide && count >= 4) {
        *reinterpret_cast<f32x4*>(s.p + i) = v;
        if (s.copy) *reinterpret_cast<bf16x4*>(s.copy + i) = __builtin_convertvector(v, bf16x4);
        return;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (q < count) {
            s.p[i + q] = v[q];
            if (s.copy) s.copy[i + q] = bf16_bits(v[q]);
        }
    }
}

// One element's step; root is the new sqrt(v).
__device__ inline void step1(const AdamwConst& c, float g, float& p, float& m, float& v,
                             float& root) {
    m = m * c.beta1 + g * c.one_beta1;
    v = v * c.beta2 + g * g * c.one_beta2;
    root = sqrtf(v);
    p = p * c.keep - m / (root * c.root_scale + c.eps) * c.rate;
}

__global__ __launch_bounds__(256) void zs_adamw_kernel(const Slices t, AdamwConst c, float* m,
                                                       float* v) {
    const Slice& s = t.s[find_slice(t, blockIdx.x)];
    const int64_t first = int64_t(blockIdx.x - s.first) * t.blocks_per_item * kBlock;
    const bool wide = s.flags & 2;
    for (int b = threadIdx.x >> 6; b < t.blocks_per_item; b += 4) {
        const int64_t i = first + b * kBlock + (threadIdx.x & 63) * 4;
        if (i >= s.n) break;
        const int count = s.n - i < 4 ? int(s.n - i) : 4;
        const int64_t si = s.offset + i;
        f32x4 pv = load_param4(s.p + i, wide, count), gv = load_grad4(s, i, wide, count);
        f32x4 mv = load_param4(m + si, true, count), vv = load_param4(v + si, true, count);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float pe = pv[q], me = mv[q], ve = vv[q], root;
            step1(c, gv[q], pe, me, ve, root);
            pv[q] = pe, mv[q] = me, vv[q] = ve;
        }
        store_param4(s, i, wide, count, pv);
        if (count >= 4) {
            *reinterpret_cast<f32x4*>(m + si) = mv;
            *reinterpret_cast<f32x4*>(v + si) = vv;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < count) m[si + q] = mv[q], v[si + q] = vv[q];
        }
    }
}

// ---- 8-bit states ---------------------------------------------------------------
constexpr uint32_t kOne = 0x3F800000u;
template <int SHIFT, int TOP>
struct Code {
    static constexpr uint32_t kBase = (kOne >> SHIFT) - TOP;
    __device__ static float value(uint32_t code) {
        return code ? __builtin_bit_cast(float, (code + kBase) << SHIFT) : 0.0f;
    }
    // magnitude mag >= 0 of a block of scale 1 / inv; random: SHIFT bits
    __device__ static uint32_t of(float mag, float inv, uint32_t random, int least) {
        float x = mag * inv;
        x = x > 1.0f ? 1.0f : x;
        if (!(x > 0.0f)) return 0;   // zeros, and blocks whose scale is not finite
        const int code = int((__builtin_bit_cast(uint32_t, x) + random) >> SHIFT) - int(kBase);
        return uint32_t(code < least ? least : (code > TOP ? TOP : code));
    }
};
using MCode = Code<20, 127>;
using VCode = Code<19, 255>;

// 32 pseudo-random bits of an element and a key: a multiplicative step by 2^32
// over the golden ratio, then the finaliser of murmur3 (public domain).
__device__ inline uint32_t hash32(uint32_t index, uint32_t key) {
    uint32_t h = index * 0x9E3779B9u + key;
    h ^= h >> 16;
    h *= 0x85EBCA6Bu;
    h ^= h >> 13;
    h *= 0xC2B2AE35u;
    return h ^ (h >> 16);
}

// Largest magnitude over the wavefront, as bits: non-negative floats order as
// their bits do, and NaN and infinity order above every number.
__device__ inline uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int h = 32; h >= 1; h >>= 1) {
        const uint32_t o = __shfl_xor(v, h, 64);
        v = o > v ? o : v;
    }
    return v;
}

// A block's scale and its reciprocal.
__device__ inline void scale_of(uint32_t bits, float& scale, float& inv) {
    scale = __builtin_bit_cast(float, bits);
    if (scale < 0x1p-120f) scale = 0.0f;
    inv = scale > 0.0f ? 1.0f / scale : scale;
}

__global__ __launch_bounds__(256) void zs_adamw8_kernel(const Slices t, AdamwConst c, uint8_t* mc,
                                                        float* ms, uint8_t* vc, float* vs,
                                                        uint32_t key) {
    const Slice& s = t.s[find_slice(t, blockIdx.x)];
    const int64_t first = int64_t(blockIdx.x - s.first) * t.blocks_per_item * kBlock;
    const bool wide = s.flags & 2;
    const int lane = threadIdx.x & 63;
    for (int b = threadIdx.x >> 6; b < t.blocks_per_item; b += 4) {
        const int64_t at = first + b * kBlock;   // of the block; the same in all lanes
        if (at >= s.n) break;
        const int64_t i = at + lane * 4;
        const int count = s.n - i < 4 ? (s.n > i ? int(s.n - i) : 0) : 4;
        const int64_t si = s.offset + i, blk = (s.offset + at) / kBlock;
        const float sm = ms[blk], sv = vs[blk];
        const uint32_t mr = *reinterpret_cast<const uint32_t*>(mc + si),
                       vr = *reinterpret_cast<const uint32_t*>(vc + si);
        f32x4 pv = load_param4(s.p + i, wide, count), gv = load_grad4(s, i, wide, count);
        float me[4], re[4];
        uint32_t m_top = 0, v_top = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t a = (mr >> (8 * q)) & 255, r = (vr >> (8 * q)) & 255;
            float mag = MCode::value(a & 127) * sm;
            me[q] = a & 128 ? -mag : mag;
            const float rt = VCode::value(r) * sv;
            float ve = rt * rt, pe = pv[q];
            step1(c, gv[q], pe, me[q], ve, re[q]);
            pv[q] = pe;
            if (q >= count) me[q] = re[q] = 0.0f;
            const uint32_t mb = __builtin_bit_cast(uint32_t, me[q]) & 0x7fffffffu,
                           rb = __builtin_bit_cast(uint32_t, re[q]) & 0x7fffffffu;
            m_top = mb > m_top ? mb : m_top;
            v_top = rb > v_top ? rb : v_top;
        }
        if (count > 0) store_param4(s, i, wide, count, pv);
        float m_scale, m_inv, v_scale, v_inv;
        scale_of(wave_max(m_top), m_scale, m_inv);
        scale_of(wave_max(v_top), v_scale, v_inv);
        uint32_t mo = 0, vo = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t h = hash32(uint32_t(i) + q, key);
            const uint32_t a = MCode::of(__builtin_fabsf(me[q]), m_inv, h & 0xFFFFFu, 0);
            const uint32_t r = VCode::of(re[q], v_inv, h >> 13, 1);
            mo |= (a | (me[q] < 0.0f ? 128u : 0u)) << (8 * q);
            vo |= r << (8 * q);
        }
        *reinterpret_cast<uint32_t*>(mc + si) = mo;
        *reinterpret_cast<uint32_t*>(vc + si) = vo;
        if (lane == 0) ms[blk] = m_scale, vs[blk] = v_scale;
    }
}

__global__ __launch_bounds__(256) void zs_moments8_kernel(const uint8_t* mc, const float* ms,
                                                          const uint8_t* vc, const float* vs,
                                                          int64_t n, float* m, float* v) {
    for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < n;
         i += int64_t(gridDim.x) * 1024) {
        const float sm = ms[i / kBlock], sv = vs[i / kBlock];
        const uint32_t mr = *reinterpret_cast<const uint32_t*>(mc + i),
                       vr = *reinterpret_cast<const uint32_t*>(vc + i);
        f32x4 mo, vo;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t a = (mr >> (8 * q)) & 255;
            const float mag = MCode::value(a & 127) * sm;
            const float rt = VCode::value((vr >> (8 * q)) & 255) * sv;
            mo[q] = a & 128 ? -mag : mag;
            vo[q] = rt * rt;
        }
        *reinterpret_cast<f32x4*>(m + i) = mo;
        *reinterpret_cast<f32x4*>(v + i) = vo;
    }
}

// Calls launch(slices, grid) for every batch of tensors.
template <typename Launch>
hipError_t batches(const zs_adamw_tensor* tensors, int64_t n_tensors, Launch launch) {
    const auto on = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; };
    int64_t at = 0;
    while (at < n_tensors) {
        Slices t{};
        int64_t blocks = 0, end = at;
        for (int64_t n = 0; end < n_tensors && n < kMaxTensors; ++end) {
            if (tensors[end].n == 0) continue;
            blocks += (tensors[end].n + kBlock - 1) / kBlock;
            ++n;
        }
        // a work item is 4 blocks (one a wavefront) until there are many items
        t.blocks_per_item = blocks > (int64_t(1) << 24) ? 64 : (blocks > 65536 ? 16 : 4);
        int64_t items = 0;
        for (; at < end; ++at) {
            const zs_adamw_tensor& a = tensors[at];
            if (a.n == 0) continue;
            Slice& s = t.s[t.count++];
            s.p = a.param, s.g = a.grad, s.copy = static_cast<uint16_t*>(a.copy);
            s.n = a.n, s.offset = a.state_offset, s.first = uint32_t(items);
            const bool half = a.grad_dtype == ZS_BF16;
            s.flags = (half ? 1u : 0u) |
                      (on(a.param, 16) && on(a.grad, half ? 8 : 16) && on(a.copy, 8) ? 2u : 0u);
            const int64_t size = int64_t(t.blocks_per_item) * kBlock;
            items += (a.n + size - 1) / size;
        }
        if (t.count == 0) break;
        if (items > 0x7fffffff) return hipErrorInvalidValue;
        const hipError_t err = launch(t, unsigned(items));
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_adamw(const zs_adamw_tensor* tensors, int64_t n_tensors, AdamwConst c, float* m,
                        float* v, hipStream_t stream) {
    return batches(tensors, n_tensors, [&](const Slices& t, unsigned grid) {
        zs_adamw_kernel<<<grid, 256, 0, stream>>>(t, c, m, v);
        return hipGetLastError();
    });
}

hipError_t launch_adamw8(const zs_adamw_tensor* tensors, int64_t n_tensors, AdamwConst c,
                         uint8_t* mc, float* ms, uint8_t* vc, float* vs, uint32_t key,
                         hipStream_t stream) {
    return batches(tensors, n_tensors, [&](const Slices& t, unsigned grid) {
        zs_adamw8_kernel<<<grid, 256, 0, stream>>>(t, c, mc, ms, vc, vs, key);
        return hipGetLastError();
    });
}

hipError_t launch_moments8(const uint8_t* mc, const float* ms, const uint8_t* vc, const float* vs,
                           int64_t n, float* m, float* v, hipStream_t stream) {
    const int64_t want = (n + 1023) / 1024;
    zs_moments8_kernel<<<unsigned(want < 65536 ? want : 65536), 256, 0, stream>>>(mc, ms, vc, vs, n,
                                                                                  m, v);
    return hipGetLastError();
}

}  // namespace zs
