// Weight gradients of the grouped products, gfx950:
// grad_w[g] = sum over the rows i of group g of x[i]^T grad_y[i].
//
// The summed index is the row, so both operands lie in LDS in sum form and are
// read transposed.  A workgroup forms a BA x BN tile of one piece (at most
// `piece` rows) of one group.  A group of one piece is written at once; the
// pieces of a longer one leave fp32 partial sums that a second kernel adds in
// order.
//
// Narrow weights (one tile, which the wavefronts also hold as fragments): the
// same pass forms grad_x[i] = grad_y[i] w[g]^T from the rows of grad_y that lie in
// LDS for the weight gradient, so that they are read once.
//
// Measured on MI355X:
//  - 647170 rows, 14 uneven groups of 16, 32 -> 96, fp32, perm, both gradients:
//    100 us and 5 us for the partial sums, 3.9 TB/s of the 417 MB that have to move
//    (81 us at a copy's rate); the weight gradient alone 66 us, at a copy's rate.
//    The fp32 matrix instructions (48 a wavefront and stage) are 50 us of it and
//    overlap the loads only in part.
//  - 8191 rows, 14 uneven groups of 16, 776 x 1160, bf16: 48 us and 7 us for the
//    partial sums, matrix cores busy 22 % of the time.  Bound by the start and end of
//    its short work items (7 stages on average, two and a half rounds of them) and by
//    what the longest group leaves.
//  - 16384 rows, one group, 4096 x 4096, bf16: 635 us, 865 TFLOP/s; two transposed
//    LDS reads feed each matrix instruction's operand.
#include "zs_block_internal.h"
#include "zs_launch.h"
#include "zs_tile.h"

namespace zs {

namespace {

template <typename T>
struct WgParams {
    const T* x;
    const T* gy;
    T* gw;
    float* partial;
    const int32_t* offsets;
    const int32_t* perm;
    int64_t ldx, ldg, n_rows, n_groups, piece;
    int k, n, k_tiles, n_tiles;
    // both gradients at once
    const T* w;
    T* gx;
    int64_t ldw, w_group;
    bool spread;   // each XCD takes an eighth of every piece's tiles
    uint32_t first, grid;   // this launch's first workgroup, the workgroups of all launches
};

__device__ inline int64_t clamp_offset(const int32_t* offsets, int64_t v, int64_t n_rows) {
    const int64_t o = offsets[v];
    return o < 0 ? 0 : (o > n_rows ? n_rows : o);
}

// Where the partial sums of a cut group that starts at position `start` begin: a
// group of c > piece rows has ceil(c / piece) <= floor(2 c / piece) pieces, and
// floor(2 (a + c) / piece) >= floor(2 a / piece) + floor(2 c / piece), so the
// pieces of cut groups never meet and end by floor(2 n_rows / piece).
__device__ inline int64_t first_piece(int64_t start, int64_t piece) { return 2 * start / piece; }

constexpr int kIndexRows = 1024;   // row indices kept in LDS at a time

// VEC as in the grouped products.  BOTH: grad_x too; k <= BA and n <= BN.
template <typename T, int BA, int BN, int WA, int WN, int KB, int S, bool VEC, bool BOTH>
__global__ __launch_bounds__(WA * WN * 64) void zs_wgrad_kernel(const WgParams<T> p) {
    constexpr int kWaves = WA * WN;
    constexpr int E = 16 / sizeof(T);
    constexpr int BR = KB / sizeof(T);    // rows of a stage
    constexpr int LN = pow2_at_least(BN);
    constexpr int kABytes = BA * KB, kBytes = kABytes + LN * KB;
    constexpr int IA = BA * KB / 1024 / kWaves, IB = LN * KB / 1024 / kWaves;
    constexpr int AT = BA / WA / 16, NT = BN / WN / 16;
    static_assert(IA >= 1 && IB >= 1 && AT >= 1 && NT >= 1, "tile too small for its wavefronts");
    extern __shared__ __align__(16) char lds[];
    __shared__ int32_t index[kIndexRows];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // BOTH: groups -1 and n_groups are the rows of no group, whose grad_x is zero
    const auto start = [&](int64_t v) -> int64_t {
        if (BOTH && v == 0) return 0;
        if (BOTH && v == p.n_groups + 2) return p.n_rows;
        return clamp_offset(p.offsets, BOTH ? v - 1 : v, p.n_rows);
    };
    const auto least = [&](int64_t v) { return BOTH && (v == 0 || v == p.n_groups + 1) ? 0 : 1; };
    const TileOf tile = find_work(p.first + blockIdx.x, p.grid, p.k_tiles * p.n_tiles, p.spread,
                                  p.n_groups + (BOTH ? 2 : 0), p.piece, start, least);
    if (tile.group < 0) return;
    const int in_slot = __builtin_amdgcn_readfirstlane(tile.sub);
    const int a0 = in_slot / p.n_tiles * BA, n0 = in_slot % p.n_tiles * BN;
    const int group = __builtin_amdgcn_readfirstlane(tile.group) - (BOTH ? 1 : 0);
    if (BOTH && (group < 0 || group >= p.n_groups)) {
        for (int64_t i = threadIdx.x; i < (tile.end - tile.begin) * p.k; i += kWaves * 64) {
            const int64_t pos = tile.begin + i / p.k;
            const int64_t r = p.perm ? p.perm[pos] : pos;
            if (r >= 0 && r < p.n_rows) p.gx[r * p.k + i % p.k] = T(0);
        }
        return;
    }

    f32x4 acc[AT][NT];
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const int wa = wave / WN, wn = wave % WN;

    // this lane's chunks of a stage: row within the stage, first kept index
    constexpr int kALanes = BA * int(sizeof(T)) / 16, kBLanes = LN * int(sizeof(T)) / 16;
    int ar[IA], ac[IA], br[IB], bc[IB];
#pragma unroll
    for (int i = 0; i < IA; ++i) {
        const int chunk = (wave * IA + i) * 64 + lane;
        ar[i] = chunk / kALanes;
        ac[i] = a0 + ((chunk % kALanes) ^ sum_swizzle<T, BA>(ar[i])) * E;
    }
#pragma unroll
    for (int i = 0; i < IB; ++i) {
        const int chunk = (wave * IB + i) * 64 + lane;
        br[i] = chunk / kBLanes;
        const int c = ((chunk % kBLanes) ^ sum_swizzle<T, LN>(br[i])) * E;
        bc[i] = c < BN ? n0 + c : p.n;
    }
    const int rows = int(tile.end - tile.begin);
    const int stages = (rows + BR - 1) / BR;
    // rows of the stages from `first` on (a multiple of kIndexRows), -1 behind the end
    const auto fill = [&](int first) {
        for (int i = threadIdx.x; i < kIndexRows && first + i < stages * BR; i += kWaves * 64) {
            int64_t r = -1;
            if (first + i < rows) {
                const int64_t pos = tile.begin + first + i;
                r = p.perm ? p.perm[pos] : pos;
                if (r < 0 || r >= p.n_rows) r = -1;
            }
            index[i] = int32_t(r);
        }
    };
    const auto load = [&](int stage, char* buf) {
        const int at = stage * BR % kIndexRows;
        // VEC: straight to LDS, row offsets of 32-bit strides; otherwise through
        // registers, all loads first
        u32x4 held[VEC ? 1 : IA + IB];
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            const int32_t r = index[at + ar[i]];
            const bool in = r >= 0 && ac[i] < p.k;
            if constexpr (VEC) {
                const T* src = p.x + uint64_t(uint32_t(r)) * uint32_t(p.ldx) + ac[i];
                load_to_lds(in ? static_cast<const void*>(src) : zero_chunk,
                            lds_offset(buf + (wave * IA + i) * 1024));
            } else {
                held[i] = load_partial(p.x + r * p.ldx + ac[i], in ? p.k - ac[i] : 0);
            }
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            const int32_t r = index[at + br[i]];
            const bool in = r >= 0 && bc[i] < p.n;
            if constexpr (VEC) {
                const T* src = p.gy + uint64_t(uint32_t(r)) * uint32_t(p.ldg) + bc[i];
                load_to_lds(in ? static_cast<const void*>(src) : zero_chunk,
                            lds_offset(buf + kABytes + (wave * IB + i) * 1024));
            } else {
                held[IA + i] = load_partial(p.gy + r * p.ldg + bc[i], in ? p.n - bc[i] : 0);
            }
        }
        if constexpr (!VEC) {
#pragma unroll
            for (int i = 0; i < IA; ++i)
                *reinterpret_cast<u32x4*>(buf + (wave * IA + i) * 1024 + lane * 16) = held[i];
#pragma unroll
            for (int i = 0; i < IB; ++i)
                *reinterpret_cast<u32x4*>(buf + kABytes + (wave * IB + i) * 1024 + lane * 16) =
                    held[IA + i];
        }
    };
    // BOTH: a wavefront forms grad_x of 16 of a stage's rows, in fp32 (stages of 32
    // rows) half of their columns; its fragments of w have the columns as the fast
    // index (in bf16 in pairs of tiles whose columns alternate by four, so that a
    // lane's results of a pair are eight neighbours) and n as the summed one
    constexpr int RT = BR / 16, KS = kWaves / RT, XT = BA / 16 / KS, NC = BN * int(sizeof(T)) / 64;
    static_assert(!BOTH || (RT * KS == kWaves && XT >= 1), "wavefronts do not cover a stage");
    const int rt = wave % RT, x0 = wave / RT * XT;
    const auto column = [&](int t, int i) {
        if (sizeof(T) == 4) return (x0 + t) * 16 + i;
        return (t >> 1) * 32 + (i >> 2) * 8 + (t & 1) * 4 + (i & 3);
    };
    typename Frag<T>::V w[BOTH ? XT : 1][BOTH ? NC : 1];
    int32_t even_row = -1, odd_row = -1;   // this lane's row of even and odd stages
    if constexpr (BOTH) {
#pragma unroll
        for (int t = 0; t < XT; ++t)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = column(t, lane & 15), n = (c * 4 + (lane >> 4)) * E;
                const T* from = p.w + group * p.w_group + k * p.ldw + n;
                w[t][c] = __builtin_bit_cast(typename Frag<T>::V,
                                             load_partial(from, k < p.k ? p.n - n : 0));
            }
    }
    // a stage's loads, with the row indices they need in LDS
    const auto issue = [&](int stage, char* buf) {
        if (stage * BR % kIndexRows == 0) {
            tile_barrier();   // every wavefront is done with the indices there
            fill(stage * BR);
            tile_barrier();
        }
        if constexpr (BOTH) {
            const int32_t r = index[stage * BR % kIndexRows + rt * 16 + (lane & 15)];
            even_row = stage & 1 ? even_row : r;
            odd_row = stage & 1 ? r : odd_row;
        }
        load(stage, buf);
    };
    const auto rows_of_x = [&](int stage, const char* at) {
        if constexpr (BOTH) {
            f32x4 x[XT];
#pragma unroll
            for (int t = 0; t < XT; ++t) x[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const auto g = read_rows_of_sum<T, LN>(at + kABytes, rt, c, lane);
#pragma unroll
                for (int step = 0; step < mma_steps<T>(); ++step)
#pragma unroll
                    for (int t = 0; t < XT; ++t) x[t] = mma_step(w[t][c], g, x[t], step);
            }
            wait_loads<0>();   // the next stage's, before the stores
            const int64_t r = stage & 1 ? odd_row : even_row;
            if (r < 0) return;
            T* to = p.gx + r * p.k;
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int t = 0; t < XT; ++t) {
                    const int k = (x0 + t) * 16 + 4 * (lane >> 4);
                    if (k < p.k) store4(to + k, x[t]);
                }
            } else {
#pragma unroll
                for (int t = 0; t < XT; t += 2) {
                    const int k = t * 16 + 8 * (lane >> 4);
                    const bf16x4 lo = __builtin_convertvector(x[t], bf16x4),
                                 hi = __builtin_convertvector(x[t + 1], bf16x4);
                    if (k < p.k)
                        *reinterpret_cast<bf16x8*>(to + k) =
                            __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                }
            }
        }
    };
    product_loop<T, AT, NT, KB, S, kBytes, IA + IB, BOTH>(
        stages, lds, acc, issue,
        [&](const char* at, int i, int s) { return read_sum_frag<T, BA>(at, wa * AT + i, s, lane); },
        [&](const char* at, int j, int s) {
            return read_sum_frag<T, LN>(at + kABytes, wn * NT + j, s, lane);
        },
        rows_of_x);

    const bool whole = tile.tiles <= 1;   // the group's only piece
    const bool wide = p.n % 4 == 0 && reinterpret_cast<uintptr_t>(p.gw) % 16 == 0;
    const int64_t slot = first_piece(clamp_offset(p.offsets, group, p.n_rows), p.piece) + tile.index;
    float* part = p.partial + slot * int64_t(p.k) * p.n;
    T* out = p.gw + group * int64_t(p.k) * p.n;
#pragma unroll
    for (int i = 0; i < AT; ++i) {
        const int a = a0 + (wa * AT + i) * 16 + (lane & 15);
        if (a >= p.k) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = n0 + (wn * NT + j) * 16 + 4 * (lane >> 4);
            const int64_t at = int64_t(a) * p.n + n;
            if (wide && n + 4 <= p.n) {
                if (whole)
                    store4(out + at, acc[i][j]);
                else
                    store4(part + at, acc[i][j]);
            } else if (whole) {
                store_partial4(out + at, acc[i][j], p.n - n);
            } else {
                store_partial4(part + at, acc[i][j], p.n - n);
            }
        }
    }
}

// Adds the partial sums of groups that were cut.  Up to 16 pieces: each thread
// adds them for four outputs of its own.  More: 64 outputs at a time, each of a
// workgroup's 16 rows of 16 lanes adds every 16th piece, four outputs a lane, and
// the 16 sums are added in order.  Few workgroups a group (kSumBlocks), because
// those of groups that were not cut have nothing to do: one for every 64 outputs
// of 16 groups of 776 x 1160 took 63 us, nearly all of it to start them.
constexpr int kSumBlocks = 256;

template <typename T>
__global__ __launch_bounds__(256) void zs_wgrad_sum_kernel(const WgParams<T> p) {
    __shared__ float sums[16][68];
    const int64_t kn = int64_t(p.k) * p.n;
    const int64_t g = blockIdx.y;
    const int64_t a = clamp_offset(p.offsets, g, p.n_rows),
                  b = clamp_offset(p.offsets, g + 1, p.n_rows);
    if (b - a <= p.piece) return;
    const int pieces = int((b - a + p.piece - 1) / p.piece);
    const float* from = p.partial + first_piece(a, p.piece) * kn;
    T* out = p.gw + g * kn;
    if (pieces <= 16 && kn % 4 == 0) {
        const bool wide = reinterpret_cast<uintptr_t>(p.gw) % 16 == 0;
        for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; i < kn;
             i += int64_t(gridDim.x) * 1024) {
            f32x4 s = {0, 0, 0, 0};
#pragma unroll 4
            for (int j = 0; j < pieces; ++j)
                s += *reinterpret_cast<const f32x4*>(from + j * kn + i);
            if (wide)
                store4(out + i, s);
            else
#pragma unroll
                for (int q = 0; q < 4; ++q) out[i + q] = T(s[q]);
        }
        return;
    }
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    for (int64_t first = int64_t(blockIdx.x) * 64; first < kn; first += int64_t(gridDim.x) * 64) {
        const int64_t i = first + col * 4;
        f32x4 s = {0, 0, 0, 0};
        if (kn % 4 == 0 && i < kn) {
#pragma unroll 4
            for (int j = row; j < pieces; j += 16)
                s += *reinterpret_cast<const f32x4*>(from + j * kn + i);
        } else {
            for (int j = row; j < pieces; j += 16)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (i + q < kn) s[q] += from[j * kn + i + q];
        }
        *reinterpret_cast<f32x4*>(&sums[row][col * 4]) = s;
        __syncthreads();
        const int64_t o = first + threadIdx.x;
        if (threadIdx.x < 64 && o < kn) {
            float t = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) t += sums[r][threadIdx.x];
            out[o] = T(t);
        }
        __syncthreads();
    }
}

template <typename T, int BA, int BN, bool VEC, bool BOTH = false>
hipError_t run(WgParams<T> p, hipStream_t stream) {
    constexpr int S = 2, KB = 128, BR = KB / sizeof(T);
    p.k_tiles = (p.k + BA - 1) / BA, p.n_tiles = (p.n + BN - 1) / BN;
    // below that an eighth of a tile's items is too coarse a share
    p.spread = p.k_tiles * p.n_tiles >= 16 && p.n_groups <= kCountedGroups;
    const int64_t slots = p.n_rows / p.piece + p.n_groups + (BOTH ? 2 : 0);
    const int64_t grid = work_grid(slots, int64_t(p.k_tiles) * p.n_tiles, p.spread);
    if (grid > 0x7fffffff) return hipErrorInvalidValue;   // gradients above 288 GB
    p.grid = uint32_t(grid);
    const int64_t longest = p.piece < p.n_rows ? p.piece : p.n_rows;
    const int stages = int((longest + BR - 1) / BR);
    const int bytes = (stages < 1 ? 1 : stages < S ? stages : S) * (BA + pow2_at_least(BN)) * KB;
    auto* kernel = zs_wgrad_kernel<T, BA, BN, 2, 2, KB, S, VEC, BOTH>;
    if (bytes + 4 * kIndexRows > 65536) {
        const hipError_t err = hipFuncSetAttribute(
            reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (err != hipSuccess) return err;
    }
    return launch_ranges(grid, 256, [&](int64_t first, int64_t count) {
        p.first = uint32_t(first);
        kernel<<<dim3(unsigned(count)), 256, bytes, stream>>>(p);
        return hipGetLastError();
    });
}

template <typename T, int BA, bool BOTH>
hipError_t by_n(const WgParams<T>& p, hipStream_t stream) {
    switch (tile_side(p.n, true)) {
        case 128: return run<T, BA, 128, true, BOTH>(p, stream);
        case 96: return run<T, BA, 96, true, BOTH>(p, stream);
        case 64: return run<T, BA, 64, true, BOTH>(p, stream);
        default: return run<T, BA, 32, true, BOTH>(p, stream);
    }
}

// Whether the operands' 16-byte chunks start on 16 bytes, strides fit 32 bits.
bool vectors(const WgradArgs& a, bool bf16) {
    const int e = bf16 ? 8 : 4;
    const auto on16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    return on16(a.x) && a.ldx % e == 0 && a.k % e == 0 && on16(a.gy) && a.ldg % e == 0 &&
           a.n % e == 0 && a.ldx <= INT32_MAX && a.ldg <= INT32_MAX;
}

template <typename T>
hipError_t dispatch(const WgradArgs& a, hipStream_t stream) {
    WgParams<T> p{static_cast<const T*>(a.x), static_cast<const T*>(a.gy), static_cast<T*>(a.gw),
                  a.partial, a.offsets, a.perm, a.ldx, a.ldg, a.n_rows, a.n_groups, a.piece,
                  a.k, a.n, 0, 0, static_cast<const T*>(a.w), static_cast<T*>(a.gx), a.ldw,
                  a.w_group, false, 0, 0};
    const bool vec = vectors(a, sizeof(T) == 2);
    hipError_t err;
    const int side = tile_side(a.k, false);
    if (!vec && a.k > 64 && a.n > 64)
        err = run<T, 128, 128, false>(p, stream);
    else if (!vec)
        err = run<T, 64, 64, false>(p, stream);
    else if (a.gx)
        err = side == 64 ? by_n<T, 64, true>(p, stream) : by_n<T, 32, true>(p, stream);
    else if (side == 128)
        err = by_n<T, 128, false>(p, stream);
    else if (side == 64)
        err = by_n<T, 64, false>(p, stream);
    else
        err = by_n<T, 32, false>(p, stream);
    if (err != hipSuccess || a.piece > a.n_rows) return err;
    const int64_t kn = int64_t(a.k) * a.n;
    for (int64_t g0 = 0; g0 < a.n_groups; g0 += 65535) {   // grid.y limit
        WgParams<T> q = p;
        q.offsets += g0;
        q.gw += g0 * kn;
        const int64_t ng = a.n_groups - g0 < 65535 ? a.n_groups - g0 : 65535;
        const int64_t bx = (kn + 63) / 64;
        zs_wgrad_sum_kernel<T><<<dim3(unsigned(bx < kSumBlocks ? bx : kSumBlocks), unsigned(ng)),
                                 256, 0, stream>>>(q);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

WgradPlan plan_wgrad(int64_t n_rows, int64_t n_groups, int64_t k, int64_t n, bool bf16) {
    const int64_t ka = tile_side(k, false), nb = tile_side(n, true);
    const int64_t tiles = ((k + ka - 1) / ka) * ((n + nb - 1) / nb);
    // One round of workgroups: rows x tiles spread evenly over as many as run at
    // once (LDS for two stages each, 160 KiB a compute unit).  Shorter pieces cost
    // more partial sums (a tile in fp32, written and read), longer ones leave
    // compute units idle behind the longest group.
    const int64_t lds = 2 * (ka + pow2_at_least(int(nb))) * 128 + 4 * kIndexRows;
    const int64_t want = 256 * (163840 / lds), step = bf16 ? 64 : 32;
    int64_t piece = (n_rows * tiles / want + step - 1) / step * step;
    if (piece < 256) piece = 256;
    if (piece >= n_rows) return WgradPlan{n_rows + 1, 0};
    return WgradPlan{piece, size_t((2 * n_rows / piece + 1) * k * n * 4)};
}

bool both_gradients(const WgradArgs& a, bool bf16) {
    return a.k <= 64 && a.n <= 128 && vectors(a, bf16) &&
           reinterpret_cast<uintptr_t>(a.gx) % 16 == 0;
}

hipError_t launch_wgrad(const WgradArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, stream) : dispatch<float>(a, stream);
}

}  // namespace zs
