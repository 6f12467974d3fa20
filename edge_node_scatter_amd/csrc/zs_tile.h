// LDS tiles and matrix-core fragments shared by the grouped products and their
// weight gradient (gfx950).
//
// A product stage covers 128 bytes of the summed index: 32 fp32 or 64 bf16
// steps.  Tiles lie in LDS in 16-byte chunks, in one of two forms:
//   row form ("R"): one tile row per kept index (a row of x, a column of y),
//     the summed index contiguous, 128 bytes a row;
//   sum form ("S"): one tile row per summed index, the kept index contiguous
//     (weights stored [k][n], and both operands of the weight gradient).
// Both forms are 128 * (kept indices) bytes.  Chunks are permuted within their
// row (XOR with a function of the row) so that a fragment's reads fall on
// different banks.
//
// mma16 multiplies 16 x 16 output tiles: lane l holds kept index l % 16 of
// both operands and, in the sub-stage of 64 bytes, the summed indices of its
// 16-byte share l / 16.  fp32 uses four 16x16x4 steps whose summed indices are
// 4 (l / 16) + step on both sides, so that a lane's share is contiguous too;
// the order of the fp32 sum is then fixed but not increasing.
// The first operand gives the output's fast index: a lane's four results are
// consecutive there.
#pragma once

#include "zs_internal.h"

namespace zs {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

constexpr int kStageBytes = 128;

// 16 bytes of zeros that lanes outside an operand load instead.
static __device__ __align__(16) const uint32_t zero_chunk[4] = {0, 0, 0, 0};

__device__ inline uint32_t lds_offset(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) const void*)(p)));
}

// 16 bytes per lane from global memory to LDS at lds + 16 * lane (lds uniform
// over the wavefront), past the registers.  Completion is counted in vmcnt;
// wait_loads() before the barrier that publishes the tile.  Inline assembly
// because the compiler otherwise drains all such loads before every transposed
// LDS read, whichever buffer it reads.  The instruction has no output registers,
// and m0 is otherwise unused here (gfx9 LDS accesses do not read it).
__device__ inline void load_to_lds(const void* g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds), "v"(g)
                 : "memory");
}
__device__ inline void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <typename T>
struct Frag;
template <>
struct Frag<float> {
    using V = f32x4;
};
template <>
struct Frag<__bf16> {
    using V = bf16x8;
};

__device__ inline f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ inline f32x4 mma16(f32x4 a, f32x4 b, f32x4 acc) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
    return acc;
}

// ---- row form -------------------------------------------------------------
__device__ inline int row_swizzle(int row) { return (row >> 1) & 7; }

// Fragment of tile rows 16 t .. 16 t + 15, sub-stage s.
template <typename T>
__device__ inline typename Frag<T>::V read_row_frag(const char* tile, int t, int s, int lane) {
    const int row = t * 16 + (lane & 15);
    const int chunk = (s * 4 + (lane >> 4)) ^ row_swizzle(row);
    return *reinterpret_cast<const typename Frag<T>::V*>(tile + row * kStageBytes + chunk * 16);
}

// ---- sum form, W kept indices per row ---------------------------------------
template <typename T, int W>
__device__ inline int sum_swizzle(int k) {
    if (sizeof(T) == 4) return 4 * ((k >> 2) & (W / 16 >= 4 ? 3 : W / 16 - 1));
    constexpr int pairs = W / 16;   // 32-byte pairs of chunks in a row
    return 2 * (((k & 3) | ((k >> 1) & 4)) & (pairs - 1));
}

// bf16: two transposed LDS reads; in each, 16 lanes read 4 rows of 16 kept
// indices and lane i receives kept index i of the 4 rows.
template <int W>
__device__ inline bf16x8 read_sum_frag_bf16(const char* tile, int t, int s, int lane) {
    const int i = lane & 15;
    union {
        i16x4 h[2];
        bf16x8 v;
    } u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int k = s * 32 + 8 * (lane >> 4) + 4 * j + (i >> 2);
        const int chunk = (t * 2 + ((i & 3) >> 1)) ^ sum_swizzle<__bf16, W>(k);
        const char* p = tile + k * (W * 2) + chunk * 16 + (i & 1) * 8;
        u.h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4*)(p));
    }
    return u.v;
}
template <int W>
__device__ inline f32x4 read_sum_frag_f32(const char* tile, int t, int s, int lane) {
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = s * 16 + 4 * (lane >> 4) + j;
        const int n = t * 16 + (lane & 15);
        const int chunk = (n >> 2) ^ sum_swizzle<float, W>(k);
        v[j] = *reinterpret_cast<const float*>(tile + k * (W * 4) + chunk * 16 + (n & 3) * 4);
    }
    return v;
}
template <typename T, int W>
__device__ inline typename Frag<T>::V read_sum_frag(const char* tile, int t, int s, int lane) {
    if constexpr (sizeof(T) == 2)
        return read_sum_frag_bf16<W>(tile, t, s, lane);
    else
        return read_sum_frag_f32<W>(tile, t, s, lane);
}

// Up to 16 bytes of elements, `count` of them valid (others zero), loaded one
// by one: operands whose rows do not start on 16 bytes.
template <typename T>
__device__ inline u32x4 load_partial(const T* p, int count) {
    constexpr int E = 16 / sizeof(T);
    union {
        T e[E];
        u32x4 v;
    } u;
    u.v = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (j < count) u.e[j] = p[j];
    return u.v;
}

// ---- ragged groups ------------------------------------------------------------
// Tiles of ragged groups without a prefix sum over them: group v, which starts
// at sorted position e(v), owns the tile slots from e(v) / step + v up to the
// next group's.  That many slots always hold its ceil(rows / step) tiles, slots
// increase with v, and all groups together have n_rows / step + groups of
// them, so a grid of that size can be launched without reading the offsets
// on the host; a slot without rows ends at once.
struct TileOf {
    int64_t begin, end;   // sorted positions of the tile
    int64_t group_end;
    int group;            // -1: no tile
    int index;            // tile number within the group
    int tiles;            // tiles of the group (0: empty group)
};

// start(v), v = 0 .. count: the groups' clamped boundaries.  64 boundaries are
// probed at a time, one per lane.
template <typename Start>
__device__ inline TileOf find_tile(int64_t slot, int64_t count, int64_t step, Start start) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = count;
    while (hi - lo > 1) {
        const int64_t stride = (hi - lo + 63) / 64;
        const int64_t v = lo + lane * stride;
        const bool below = v < hi && start(v) / step + v <= slot;
        const int n = __popcll(__ballot(below));
        const int64_t next = lo + (n > 0 ? n - 1 : 0) * stride;
        hi = next + stride < hi ? next + stride : hi;
        lo = next;
    }
    TileOf t;
    const int64_t a = start(lo), b = start(lo + 1);
    const int64_t rel = slot - (a / step + lo);
    t.tiles = b > a ? int((b - a + step - 1) / step) : 0;
    t.begin = a + rel * step;
    t.end = t.begin + step < b ? t.begin + step : b;
    t.group_end = b;
    t.index = int(rel);
    t.group = rel >= 0 && (t.begin < b || rel == 0) ? int(lo) : -1;
    if (t.end < t.begin) t.end = t.begin;
    return t;
}

// Hands each XCD (workgroups go to the 8 XCDs in turn) a contiguous range of
// work items, so that neighbouring items share an L2.
__device__ inline int64_t xcd_item(int64_t id, int64_t total) {
    const int64_t per = total / 8, rest = total % 8, xcd = id % 8, i = id / 8;
    return xcd * per + (xcd < rest ? xcd : rest) + i;
}

}  // namespace zs
