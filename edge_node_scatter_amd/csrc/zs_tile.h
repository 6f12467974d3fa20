// LDS tiles and matrix-core fragments shared by the grouped products and their
// weight gradient (gfx950).
//
// A product stage covers KB = 64 or 128 bytes of the summed index (16 or 32
// fp32, 32 or 64 bf16 steps).  Tiles lie in LDS in 16-byte chunks, in one of two forms:
//   row form ("R"): one tile row per kept index (a row of x, a column of y),
//     the summed index contiguous, KB bytes a row;
//   sum form ("S"): one tile row per summed index, the kept index contiguous
//     (weights stored [k][n], and both operands of the weight gradient).
// Both forms are KB * (kept indices) bytes.  Chunks are permuted within their
// row (XOR with a function of the row) so that a fragment's reads fall on
// different banks.
//
// Matrix instructions multiply 16 x 16 output tiles: lane l holds kept index l % 16 of
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
// LDS read, whichever buffer it reads.  The instruction has no output registers.
// m0 is reserved, so a clobber list cannot name it: no kernel with these loads may
// have another use of m0 (gfx9 LDS accesses do not read it), which a test of the
// listings holds.
__device__ inline void load_to_lds(const void* g, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds), "v"(g)
                 : "memory");
}
// All but the latest N of this wavefront's loads have arrived.
template <int N>
__device__ inline void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt has 6 bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Workgroup barrier that waits for LDS accesses but leaves loads to LDS in
// flight; wait_loads() says which of those have arrived.
__device__ inline void tile_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

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

// One step of a 16 x 16 product: all of a bf16 fragment, a quarter of an fp32 one.
// The steps of several tiles are taken in turn, so that an instruction does not
// wait for the one before it.
template <typename T>
constexpr int mma_steps() {
    return sizeof(T) == 4 ? 4 : 1;
}
__device__ inline f32x4 mma_step(bf16x8 a, bf16x8 b, f32x4 acc, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ inline f32x4 mma_step(f32x4 a, f32x4 b, f32x4 acc, int step) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a[step], b[step], acc, 0, 0, 0);
}

// ---- row form -------------------------------------------------------------
// 16 rows at one chunk fall on all 64 banks.
template <int KB>
__device__ inline int row_swizzle(int row) {
    return KB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// Fragment of tile rows 16 t .. 16 t + 15, sub-stage s.
template <typename T, int KB>
__device__ inline typename Frag<T>::V read_row_frag(const char* tile, int t, int s, int lane) {
    const int row = t * 16 + (lane & 15);
    const int chunk = (s * 4 + (lane >> 4)) ^ row_swizzle<KB>(row);
    return *reinterpret_cast<const typename Frag<T>::V*>(tile + row * KB + chunk * 16);
}

// ---- sum form, W kept indices per row ---------------------------------------
// Spreads both kinds of read over the banks: the transposed reads of the summed
// index, and reads of 16 rows at one chunk (the row form of the same tile).
template <typename T, int W>
__device__ inline int sum_swizzle(int k) {
    if constexpr (sizeof(T) == 4) return 4 * ((k >> 2) & (W / 16 >= 4 ? 3 : W / 16 - 1)) | (k & 3);
    constexpr int pairs = W / 16;   // 32-byte pairs of chunks in a row
    return 2 * (((k & 3) | ((k >> 1) & 4)) & (pairs - 1)) | ((k >> 2) & 1);
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
// Row-form fragment of a sum-form tile: tile rows 16 t .. 16 t + 15 as kept
// indices, the 64 bytes s of their columns as summed ones.
template <typename T, int W>
__device__ inline typename Frag<T>::V read_rows_of_sum(const char* tile, int t, int s, int lane) {
    const int row = t * 16 + (lane & 15);
    const int chunk = (s * 4 + (lane >> 4)) ^ sum_swizzle<T, W>(row);
    return *reinterpret_cast<const typename Frag<T>::V*>(tile + row * (W * int(sizeof(T))) +
                                                         chunk * 16);
}
template <typename T, int W>
__device__ inline typename Frag<T>::V read_sum_frag(const char* tile, int t, int s, int lane) {
    if constexpr (sizeof(T) == 2)
        return read_sum_frag_bf16<W>(tile, t, s, lane);
    else
        return read_sum_frag_f32<W>(tile, t, s, lane);
}

// 16 bytes of elements whose first `count` exist (the others zero), from any
// element's address: one unaligned access where all exist.
template <typename T>
__device__ inline u32x4 load_partial(const T* p, int count) {
    constexpr int E = 16 / sizeof(T);
    union {
        T e[E];
        u32x4 v;
    } u;
    u.v = u32x4{0, 0, 0, 0};
    if (count >= E) {
        __builtin_memcpy(&u.v, p, 16);
    } else if (count > 0) {
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (j < count) u.e[j] = p[j];
    }
    return u.v;
}
// Four results to any element's address, the first `count` of them.
template <typename T>
__device__ inline void store_partial4(T* p, f32x4 v, int count) {
    const T e[4] = {T(v[0]), T(v[1]), T(v[2]), T(v[3])};
    if (count >= 4) {
        __builtin_memcpy(p, e, 4 * sizeof(T));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < count) p[j] = e[j];
    }
}

template <typename T>
__device__ inline void store4(T* p, f32x4 v) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4*>(p) = v;
    } else {
        *reinterpret_cast<bf16x4*>(p) = __builtin_convertvector(v, bf16x4);
    }
}

// The products of one stage; read_a(buf, i, s) and read_b(buf, j, s) read the
// fragments of its sub-stage s.
template <typename T, int MT, int NT, int KB, typename ReadA, typename ReadB>
__device__ inline void multiply_stage(const char* at, f32x4 (&acc)[MT][NT], ReadA read_a,
                                      ReadB read_b) {
    using V = typename Frag<T>::V;
#pragma unroll
    for (int s = 0; s < KB / 64; ++s) {
        V a[MT], b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = read_b(at, j, s);
#pragma unroll
        for (int i = 0; i < MT; ++i) a[i] = read_a(at, i, s);
#pragma unroll
        for (int step = 0; step < mma_steps<T>(); ++step)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = mma_step(b[j], a[i], acc[i][j], step);
    }
}

// The product loop over `stages` stages, S buffers of kBytes deep.  issue(i, buf)
// starts the loads of stage i (kLoads per wavefront); also(i, buf) does what else
// a stage is for.  One barrier a stage: it publishes the stage and says that every
// wavefront is done with the one before, whose buffer the next loads fill.
// (Reading the fragments of the next sub-stage ahead, across the barrier, was no
// faster in the products and slower in the weight gradient, whose transposed reads
// then crowd its registers: 16384 x 4096 x 4096 in bf16 495 us either way, its
// weight gradient 680 and 775.)
//
// LATE (S = 2): also() stores, and stores count as loads do; so it is also()
// that waits for the next stage's loads, before it stores, and the stores have
// until the next stage's end.
template <typename T, int MT, int NT, int KB, int S, int kBytes, int kLoads, bool LATE,
          typename Issue, typename ReadA, typename ReadB, typename Also>
__device__ inline void product_loop(int stages, char* lds, f32x4 (&acc)[MT][NT], Issue issue,
                                    ReadA read_a, ReadB read_b, Also also) {
    if (stages <= 0) return;
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (i < stages) issue(i, lds + i * kBytes);
    int cur = 0;
    for (int stage = 0; stage < stages; ++stage) {
        // `stage` has arrived when at most the S - 2 stages behind it are in flight
        static_assert(!LATE || S == 2, "also() waits for one stage");
        if (!LATE || stage == 0) {
            if (stage + S - 1 <= stages)
                wait_loads<(S - 2) * kLoads>();
            else
                wait_loads<0>();
        }
        tile_barrier();
        const char* at = lds + cur * kBytes;
        if (stage + S - 1 < stages) issue(stage + S - 1, lds + (cur == 0 ? S - 1 : cur - 1) * kBytes);
        cur = cur + 1 == S ? 0 : cur + 1;
        multiply_stage<T, MT, NT, KB>(at, acc, read_a, read_b);
        also(stage, at);
    }
}

// Width of an LDS tile's rows for `v` kept indices: a wavefront's load covers whole
// rows.
constexpr int pow2_at_least(int v) { return v <= 32 ? 32 : v <= 64 ? 64 : v <= 128 ? 128 : 256; }

// Side of the tiles that cover `width`: as few tiles as sides of 128 need, as
// narrow as covers it, so that little of a tile is padding while wide operands
// are still read as few times as 128 allows.
inline int tile_side(int64_t width, bool with96) {
    const int64_t tiles = (width + 127) / 128;
    for (int s : {32, 64, 96})
        if ((s != 96 || with96) && s * tiles >= width) return s;
    return 128;
}

// A wavefront's 16 x (16 NT) results of one row of tiles in bf16, through its part
// of the LDS (16 rows of kRowBytes), so that stores write whole lines: straight from
// the accumulators a store instruction covers 32 bytes of each of 16 rows.  write()
// puts the results there, read() returns the 16-byte chunk `id` (row id / kChunks).
// Chunks are rotated within their row against bank conflicts.
template <int NT>
struct RowsOut {
    static constexpr int kRowBytes = NT * 32, kChunks = NT * 2, kTurns = NT / 2;
    static constexpr int kBytes = 16 * kRowBytes;
    static_assert(NT % 2 == 0, "a store takes 64 chunks");
    __device__ static char* at(char* lds, int row, int chunk) {
        const int turn = kRowBytes >= 256 ? row : (kRowBytes == 128 ? row >> 1 : row >> 2);
        return lds + row * kRowBytes + (chunk + turn) % kChunks * 16;
    }
    __device__ static void write(char* lds, const f32x4 (&acc)[NT], int lane) {
        const int row = lane & 15, q = lane >> 4;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            store4(reinterpret_cast<__bf16*>(at(lds, row, 2 * j + q / 2) + q % 2 * 8), acc[j]);
    }
    __device__ static u32x4 read(char* lds, int id) {
        return *reinterpret_cast<const u32x4*>(at(lds, id / kChunks, id % kChunks));
    }
};

// The first `count` values of a 16-byte chunk, to an address on 16 bytes.
template <typename T>
__device__ inline void store_partial(T* p, u32x4 v, int count) {
    constexpr int E = 16 / sizeof(T);
    if (count >= E) {
        *reinterpret_cast<u32x4*>(p) = v;
        return;
    }
    union {
        u32x4 v;
        T e[E];
    } u;
    u.v = v;
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (j < count) p[j] = u.e[j];
}

// ---- ragged groups ------------------------------------------------------------
// The tiles of ragged groups are numbered without the host reading the offsets:
// the grid holds as many workgroups as there can be tiles (one part-filled tile
// a group), each finds its own, and those behind the last end at once.
struct TileOf {
    int64_t begin, end;   // sorted positions of the tile
    int group;            // -1: no tile
    int index;            // tile number within the group
    int tiles;            // tiles of the group (0: empty group)
    int sub;              // which of the tile's `subs` work items
};

__device__ inline TileOf tile_at(int64_t v, int64_t index, int64_t step, int64_t a, int64_t b) {
    TileOf t;
    t.tiles = b > a ? int((uint32_t(b - a) + uint32_t(step) - 1) / uint32_t(step)) : 0;
    t.begin = a + index * step;
    t.end = t.begin + step < b ? t.begin + step : b;
    if (t.end < t.begin) t.end = t.begin;
    t.group = int(v);
    t.index = int(index);
    t.sub = 0;
    return t;
}

// Up to this many groups a wavefront adds up all groups' tiles, 64 at a time.
constexpr int kCountedGroups = 512;

// Workgroups for at most `tiles` tiles of `subs` work items: find_work gives an
// XCD an eighth of each of two kinds, both rounded up, or of each tile.
inline int64_t work_grid(int64_t tiles, int64_t subs, bool spread) {
    return spread ? 8 * tiles * ((subs + 7) / 8) : tiles * subs + 16;
}

// Inclusive sum over the wavefront's lanes: within rows of 16 lanes by shifts,
// then the last lane of the rows before.
__device__ inline uint32_t lane_scan(uint32_t n) {
    int v = int(n);
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // lane 15 to the next row
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // lane 31 to the upper half
    return uint32_t(v);
}

// The work of workgroup `id`: start(v), v = 0 .. count, are the groups' clamped
// boundaries; group v has a tile for each `step` of its rows, least(v) at least,
// and a tile `subs` work items.
//
// Workgroups go to the 8 XCDs in turn, so XCD x, which holds the ids x, x + 8,
// ..., gets an eighth of the full tiles' items and then an eighth of the
// part-filled tiles', each in one piece: neighbouring items share its L2, no XCD
// has more to do than another, and what is dispatched last is short.  With
// `spread` an XCD instead gets an eighth of every tile's items: for work whose
// part-filled tiles differ in length, so that the XCDs stay even (8191 rows in 16
// uneven groups, 776 x 1160 gradients in bf16: CUs busy 52 % of the time without).
// (Dealing
// out the ids of the second scheme, whose empty ones fall anywhere, left some
// XCDs a tile more than they have room for at a time: 16384 rows of 8 equal
// groups, 512 -> 512 in fp32, took 113 us instead of 83.)
//
// With more groups, group v owns the slots from start(v) / step + v up to the
// next group's: never fewer than its tiles, increasing with v, and a search over
// the boundaries, 64 probes at a time, finds a slot's group.
template <typename Start, typename Least>
__device__ inline TileOf find_work(uint32_t id, uint32_t grid, int subs, bool spread,
                                   int64_t count, int64_t step, Start start, Least least) {
    const int lane = threadIdx.x & 63;
    TileOf none{};
    none.group = -1;
    const uint32_t xcd = id % 8;
    uint32_t nth = id / 8;
    if (count <= kCountedGroups) {
        constexpr int kChunks = kCountedGroups / 64;
        const int chunks = int((count + 63) / 64);
        // of this lane's groups: first position, rows, full tiles up to it, whether
        // it has a part-filled tile
        uint32_t at[kChunks], rows[kChunks], before[kChunks];
        uint64_t part[kChunks];
        uint32_t total[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            at[c] = rows[c] = before[c] = 0;
            part[c] = 0;
            if (c >= chunks) continue;
            const int64_t v = c * 64 + lane;
            uint32_t full = 0;
            bool more = false;
            if (v < count) {
                const int64_t a = start(v), b = start(v + 1);
                at[c] = uint32_t(a);
                rows[c] = b > a ? uint32_t(b - a) : 0;
                full = rows[c] / uint32_t(step);
                more = full * uint32_t(step) < rows[c] || (rows[c] == 0 && least(v) > 0);
            }
            before[c] = total[0] + lane_scan(full);
            part[c] = __ballot(more);
            total[0] = __builtin_amdgcn_readlane(before[c], 63);
            total[1] += uint32_t(__popcll(part[c]));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t tile;
            int sub;
            if (spread) {
                const uint32_t first = uint32_t(subs) * xcd / 8,
                               mine = uint32_t(subs) * (xcd + 1) / 8 - first;
                tile = nth / mine;
                sub = int(first + nth - tile * mine);
                if (tile >= total[k]) {
                    nth -= total[k] * mine;
                    continue;
                }
            } else {
                const uint64_t items = uint64_t(total[k]) * uint32_t(subs);
                const uint64_t per = items / 8, rest = items % 8;
                const uint32_t mine = uint32_t(per) + (xcd < rest ? 1 : 0);
                if (nth >= mine) {
                    nth -= mine;
                    continue;
                }
                const uint64_t item = xcd * per + (xcd < rest ? xcd : rest) + nth;
                tile = uint32_t(item / uint32_t(subs));
                sub = int(item - uint64_t(tile) * uint32_t(subs));
            }
            uint32_t base = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (c >= chunks) continue;
                int l = -1;
                uint32_t index = 0;
                if (k == 0) {
                    if (tile < uint32_t(__builtin_amdgcn_readlane(before[c], 63))) {
                        // lanes whose groups lie before the tile's
                        l = __popcll(__ballot(before[c] <= tile));
                        index = tile - (l > 0 ? uint32_t(__builtin_amdgcn_readlane(before[c], l - 1))
                                              : base);
                    }
                    base = __builtin_amdgcn_readlane(before[c], 63);
                } else {
                    const uint32_t here = uint32_t(__popcll(part[c]));
                    if (tile < here) {
                        // the lane of the tile-th part-filled tile: it has `tile` before it
                        const uint32_t mine_before = __builtin_amdgcn_mbcnt_hi(
                            uint32_t(part[c] >> 32),
                            __builtin_amdgcn_mbcnt_lo(uint32_t(part[c]), 0));
                        l = __ffsll(__ballot(mine_before == tile && ((part[c] >> lane) & 1))) - 1;
                        index = uint32_t(__builtin_amdgcn_readlane(rows[c], l)) / uint32_t(step);
                    } else {
                        tile -= here;
                    }
                }
                if (l >= 0) {
                    const int64_t a = uint32_t(__builtin_amdgcn_readlane(at[c], l));
                    const int64_t n = uint32_t(__builtin_amdgcn_readlane(rows[c], l));
                    TileOf t = tile_at(c * 64 + l, index, step, a, a + n);
                    t.sub = sub;
                    return t;
                }
            }
        }
        return none;
    }
    const uint32_t per = grid / 8, rest = grid % 8;
    const uint32_t item = xcd * per + (xcd < rest ? xcd : rest) + nth;
    const int64_t slot = item / uint32_t(subs);
    int64_t lo = 0, hi = count;
    while (hi - lo > 1) {
        const int64_t stride = (hi - lo + 63) / 64;
        const int64_t v = lo + lane * stride;
        const bool below = v < hi && uint32_t(start(v)) / uint32_t(step) + v <= slot;
        const int n = __popcll(__ballot(below));
        const int64_t next = lo + (n > 0 ? n - 1 : 0) * stride;
        hi = next + stride < hi ? next + stride : hi;
        lo = next;
    }
    const int64_t a = start(lo);
    const int64_t index = slot - (uint32_t(a) / uint32_t(step) + lo);
    if (index < 0) return none;
    TileOf t = tile_at(lo, index, step, a, start(lo + 1));
    if (index >= (t.tiles > 0 ? t.tiles : least(lo))) return none;
    t.sub = int(item - uint32_t(slot) * uint32_t(subs));
    return t;
}

}  // namespace zs
