// Grouped products y[i] = x[i] op(w[g(i)]) for gfx950.
//
// One workgroup forms a BM x BN tile of one group's rows: x rows (gathered
// through perm) and the group's weights go through LDS in stages of KB bytes of
// k, S buffers deep, and the matrix cores accumulate in fp32.  The grid is the
// largest number of tiles the sizes allow; a workgroup finds its own from the
// offsets (zs_tile.h), so nothing is read back and one launch does it all.
//
// Measured on MI355X (a copy reaches 5.1 TB/s, library products 1.22 to 1.27
// PFLOP/s in bf16 and 150 TFLOP/s in fp32):
//  - 158002 rows, 8 uneven groups of 9, 32 -> 96, fp32, perm: 23 us, 3.5 TB/s.  Bound
//    by memory (16 us); the workgroups, few for each compute unit, load, multiply
//    (matrix cores 30 % busy) and store largely in step.  Rows streamed past weights
//    held in registers, without LDS, took 28 us.
//  - 16384 rows, 7 uneven groups of 8, 1024 -> 2048, bf16: 85 us, 808 TFLOP/s (matrix
//    cores busy 42 % of the time); one group, 4096 -> 4096: 488 us, 1127 TFLOP/s (1157
//    with weights [n][k]).  A 256 x 256 stage is 2048 cycles of matrix instructions
//    and as many of loads to LDS (a wavefront's 1 KB takes the address unit 32
//    cycles), and their overlap is not complete: matrix cores busy 53 % of the time.
//  - 96 rows, 4 groups, 64 -> 64, fp32: 4.8 us, of which most is latency: offsets,
//    row indices and operands are read one after the other.
#include <math.h>

#include "zs_block_internal.h"
#include "zs_launch.h"
#include "zs_tile.h"

namespace zs {

namespace {

template <typename T>
struct MmParams {
    const T* x;
    const T* w;
    T* y;
    const int32_t* offsets;
    const int32_t* perm;
    int64_t ldx, ldw, w_group, ldy, n_rows, n_groups;
    int k, n, n_tiles;
    uint32_t first, grid;   // this launch's first workgroup, the workgroups of all launches
};

// WT: weights stored [n][k] (row form in LDS), else [k][n] (sum form).
// VEC: the operands' chunks of 16 bytes start on 16 bytes and lie wholly
// inside or outside them, so they are loaded straight to LDS; otherwise
// elements are loaded one by one.
template <typename T, int BM, int BN, int WM, int WN, int KB, int S, bool WT, bool VEC>
__global__ __launch_bounds__(WM * WN * 64) void zs_gmm_kernel(const MmParams<T> p) {
    constexpr int kWaves = WM * WN;
    constexpr int E = 16 / sizeof(T);              // elements of a chunk
    constexpr int BK = KB / sizeof(T);
    constexpr int LN = pow2_at_least(BN);          // width of the weight tile in LDS
    constexpr int kABytes = BM * KB, kBytes = kABytes + LN * KB;
    constexpr int kRows = 1024 / KB, kChunks = KB / 16;   // of a wavefront's load, of a row
    constexpr int IA = BM / kRows / kWaves, IB = LN / kRows / kWaves;   // loads per wavefront and stage
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    static_assert(IA >= 1 && IB >= 1 && MT >= 1 && NT >= 1, "tile too small for its wavefronts");
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // groups 0 and n_groups + 1 are the rows before the first and behind the
    // last offset: they get zeros
    const auto start = [&](int64_t v) -> int64_t {
        if (v == 0) return 0;
        if (v == p.n_groups + 2) return p.n_rows;
        const int64_t o = p.offsets[v - 1];
        return o < 0 ? 0 : (o > p.n_rows ? p.n_rows : o);
    };
    const TileOf tile = find_work(p.first + blockIdx.x, p.grid, p.n_tiles, false, p.n_groups + 2, BM,
                                  start, [](int64_t) { return 0; });
    if (tile.group < 0) return;
    const int n0 = __builtin_amdgcn_readfirstlane(tile.sub) * BN;
    const int group = __builtin_amdgcn_readfirstlane(tile.group) - 1;
    const bool in_group = group >= 0 && group < p.n_groups;

    const auto row_at = [&](int m) -> int64_t {   // row of tile row m, -1 if none
        const int64_t pos = tile.begin + m;
        if (pos >= tile.end) return -1;
        if (!p.perm) return pos;
        const int64_t r = p.perm[pos];
        return r >= 0 && r < p.n_rows ? r : -1;
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const int wm = wave / WN, wn = wave % WN;

    if (in_group) {
        const T* w = p.w + group * p.w_group;
        // this lane's chunks: pointer at k = 0 (NULL outside) and first k / n
        const T* a_ptr[IA];
        int a_k[IA];
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            const int m = (wave * IA + i) * kRows + lane / kChunks;
            const int64_t r = row_at(m);
            a_k[i] = ((lane % kChunks) ^ row_swizzle<KB>(m)) * E;
            a_ptr[i] = r < 0 ? nullptr : p.x + r * p.ldx + a_k[i];
        }
        const T* b_ptr[IB];
        int b_k[IB], b_n[IB];
        constexpr int kLanes = LN * int(sizeof(T)) / 16;   // lanes of a row, sum form
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            if constexpr (WT) {
                const int c = (wave * IB + i) * kRows + lane / kChunks;
                b_k[i] = ((lane % kChunks) ^ row_swizzle<KB>(c)) * E;
                b_n[i] = n0 + c;
                b_ptr[i] = c < BN && b_n[i] < p.n ? w + int64_t(b_n[i]) * p.ldw + b_k[i] : nullptr;
            } else {
                const int chunk = (wave * IB + i) * 64 + lane;
                b_k[i] = chunk / kLanes;
                const int c = ((chunk % kLanes) ^ sum_swizzle<T, LN>(b_k[i])) * E;
                b_n[i] = n0 + c;
                b_ptr[i] = c < BN && b_n[i] < p.n ? w + int64_t(b_k[i]) * p.ldw + b_n[i] : nullptr;
            }
        }
        const int stages = (p.k + BK - 1) / BK;
        const auto read_a = [&](const char* at, int i, int s) {
            return read_row_frag<T, KB>(at, wm * MT + i, s, lane);
        };
        const auto read_b = [&](const char* at, int j, int s) {
            if constexpr (WT)
                return read_row_frag<T, KB>(at + kABytes, wn * NT + j, s, lane);
            else
                return read_sum_frag<T, LN>(at + kABytes, wn * NT + j, s, lane);
        };
        if constexpr (VEC) {
            const auto load = [&](int stage, char* buf) {
                const int k0 = stage * BK;
#pragma unroll
                for (int i = 0; i < IA; ++i) {
                    const bool in = a_ptr[i] && k0 + a_k[i] < p.k;
                    load_to_lds(in ? static_cast<const void*>(a_ptr[i] + k0) : zero_chunk,
                                lds_offset(buf + (wave * IA + i) * 1024));
                }
#pragma unroll
                for (int i = 0; i < IB; ++i) {
                    const bool in = b_ptr[i] && k0 + b_k[i] < p.k;
                    const T* src = b_ptr[i] + (WT ? int64_t(k0) : int64_t(k0) * p.ldw);
                    load_to_lds(in ? static_cast<const void*>(src) : zero_chunk,
                                lds_offset(buf + kABytes + (wave * IB + i) * 1024));
                }
            };
            product_loop<T, MT, NT, KB, S, kBytes, IA + IB, false>(
                stages, lds, acc, load, read_a, read_b, [](int, const char*) {});
        } else {
            // S stages at a time through registers, so that their loads' latency is
            // paid once: all loads, all writes to LDS, then the products (10 rows of 4
            // groups, 1001 -> 1501 with weights [n][k] in bf16: 21 us with two buffers
            // in turn, 13 with four stages at a time).  Large products keep one: their
            // compute units have other workgroups to go on with, and registers for two
            // stages leave room for fewer (16384 x 1001 -> 2047: 392 and 206 us).
            for (int first = 0; first < stages; first += S) {
                u32x4 held[S][IA + IB];
#pragma unroll
                for (int u = 0; u < S; ++u) {
                    const int k0 = (first + u) * BK;
#pragma unroll
                    for (int i = 0; i < IA; ++i) {
                        const int left = a_ptr[i] ? p.k - k0 - a_k[i] : 0;
                        held[u][i] = load_partial(a_ptr[i] + k0, left);
                    }
#pragma unroll
                    for (int i = 0; i < IB; ++i) {
                        const bool in = b_ptr[i] && k0 + b_k[i] < p.k;
                        const int left = WT ? p.k - k0 - b_k[i] : p.n - b_n[i];
                        held[u][IA + i] = load_partial(
                            b_ptr[i] + (WT ? int64_t(k0) : int64_t(k0) * p.ldw), in ? left : 0);
                    }
                }
                tile_barrier();   // every wavefront is done with the stages before
#pragma unroll
                for (int u = 0; u < S; ++u) {
                    if (u >= stages) break;   // as many buffers as stages at most
                    char* buf = lds + u * kBytes + lane * 16;
#pragma unroll
                    for (int i = 0; i < IA; ++i)
                        *reinterpret_cast<u32x4*>(buf + (wave * IA + i) * 1024) = held[u][i];
#pragma unroll
                    for (int i = 0; i < IB; ++i)
                        *reinterpret_cast<u32x4*>(buf + kABytes + (wave * IB + i) * 1024) =
                            held[u][IA + i];
                }
                tile_barrier();
                for (int u = 0; u < S && first + u < stages; ++u)
                    multiply_stage<T, MT, NT, KB>(lds + u * kBytes, acc, read_a, read_b);
            }
        }
    }

    // bf16 rows of y on 16 bytes go through LDS as whole lines (16384 x 1024 -> 2048:
    // 94 us straight from the accumulators, 85 so; 50182 x 128 -> 1328: 69 and 58).
    // fp32 stores from the accumulators fill 64 bytes of a row and are as fast.
    if constexpr (sizeof(T) == 2) {
        using Out = RowsOut<NT>;
        static_assert(kWaves * Out::kBytes <= kBytes, "results fit the buffer of one stage");
        if (p.ldy % E == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0) {
            tile_barrier();   // every wavefront is done with the operands
            char* mine = lds + wave * Out::kBytes;
            const int first_n = n0 + wn * NT * 16;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                // a row's number is below 2^31
                const int row = int(row_at((wm * MT + i) * 16 + (lane & 15)));
                Out::write(mine, acc[i], lane);
                wave_lds_sync();
#pragma unroll
                for (int t = 0; t < Out::kTurns; ++t) {
                    const int id = t * 64 + lane;
                    const int64_t r = __shfl(row, id / Out::kChunks, 64);
                    const int n = first_n + id % Out::kChunks * E;
                    if (r >= 0 && n < p.n)
                        store_partial(p.y + r * p.ldy + n, Out::read(mine, id), p.n - n);
                }
                wave_lds_sync();
            }
            return;
        }
    }
    const bool wide = p.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % (4 * sizeof(T)) == 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t r = row_at((wm * MT + i) * 16 + (lane & 15));
        if (r < 0) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = n0 + (wn * NT + j) * 16 + 4 * (lane >> 4);
            T* to = p.y + r * p.ldy + n;
            if (wide && n + 4 <= p.n)
                store4(to, acc[i][j]);
            else
                store_partial4(to, acc[i][j], p.n - n);
        }
    }
}

template <typename T, int BM, int BN, int WM, int WN, int KB, int S, bool WT, bool VEC>
hipError_t run(const GmmArgs& a, hipStream_t stream) {
    constexpr int BK = KB / sizeof(T);
    MmParams<T> p{static_cast<const T*>(a.x), static_cast<const T*>(a.w), static_cast<T*>(a.y),
                  a.offsets, a.perm, a.ldx, a.ldw, a.w_group, a.ldy, a.n_rows, a.n_groups,
                  a.k, a.n, (a.n + BN - 1) / BN, 0, 0};
    const int64_t slots = a.n_rows / BM + a.n_groups + 2;
    const int64_t grid = work_grid(slots, p.n_tiles, false);
    // at most 2^29 for the groups; more for rows only with outputs above 288 GB
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    p.grid = uint32_t(grid);
    // no more buffers than stages: short sums leave LDS for more workgroups
    const int stages = (a.k + BK - 1) / BK;
    const int bytes = (stages < S ? stages : S) * (BM + pow2_at_least(BN)) * KB;
    auto* kernel = zs_gmm_kernel<T, BM, BN, WM, WN, KB, S, WT, VEC>;
    if (bytes > 65536) {
        const hipError_t err = hipFuncSetAttribute(
            reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (err != hipSuccess) return err;
    }
    return launch_ranges(grid, WM * WN * 64, [&](int64_t first, int64_t count) {
        p.first = uint32_t(first);
        kernel<<<dim3(unsigned(count)), WM * WN * 64, bytes, stream>>>(p);
        return hipGetLastError();
    });
}

template <typename T, bool WT>
hipError_t dispatch(const GmmArgs& a, hipStream_t stream) {
    constexpr int E = 16 / sizeof(T);
    const auto on16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool vec = on16(a.x) && a.ldx % E == 0 && a.k % E == 0 && on16(a.w) && a.ldw % E == 0 &&
                     a.w_group % E == 0 && (WT || a.n % E == 0);
    const auto tiles = [&](int bm, int bn) {
        return (a.n_rows / bm + a.n_groups) * ((a.n + bn - 1) / bn);
    };
    const bool few = tiles(128, 128) < 256;
    if (!vec && !few && a.n > 64) return run<T, 128, 128, 2, 2, 128, 1, WT, false>(a, stream);
    if (!vec) return run<T, 64, 64, 2, 2, 128, 4, WT, false>(a, stream);
    // tiles too few for the compute units: smaller ones, more stages in flight
    if (few) return run<T, 32, 64, 2, 2, 128, 4, WT, true>(a, stream);
    const int bn = tile_side(a.n, true);
    if (bn == 128) {
        // bf16 with work for all compute units: tiles of 256 columns, one workgroup a
        // compute unit; of 256 rows, or of 192 where their last round of workgroups
        // leaves less idle (a group has half a tile of padding on average; of many
        // rounds the last is less than a whole one, as workgroups drift apart).
        // 16384 x 1024 -> 2048 in 7 uneven groups: 84 us with 192 rows, 95 with 256;
        // 16384 x 4096 -> 4096 in one group: 551 us with 192, 489 with 256.
        if constexpr (sizeof(T) == 2) {
            if (tiles(256, 256) >= 256) {
                const auto cost = [&](int bm) {
                    const double rows = a.n_groups == 1 ? (a.n_rows + bm - 1) / bm
                                                        : double(a.n_rows) / bm + 0.5 * a.n_groups;
                    const double rounds = rows * ((a.n + 255) / 256) / 256;
                    return bm * (rounds < 3 ? ceil(rounds) : rounds + 0.5);
                };
                if (1.05 * cost(192) < cost(256))
                    return run<T, 192, 256, 2, 4, 128, 2, WT, true>(a, stream);
                return run<T, 256, 256, 2, 4, 128, 2, WT, true>(a, stream);
            }
        }
        return run<T, 128, 128, 2, 2, 128, 2, WT, true>(a, stream);
    }
    if (bn == 96) return run<T, 128, 96, 4, 1, 128, 2, WT, true>(a, stream);
    if (bn == 64) return run<T, 128, 64, 4, 1, 128, 2, WT, true>(a, stream);
    return run<T, 128, 32, 4, 1, 128, 2, WT, true>(a, stream);
}

}  // namespace

hipError_t launch_gmm(const GmmArgs& a, bool bf16, bool w_transposed, hipStream_t stream) {
    if (bf16)
        return w_transposed ? dispatch<__bf16, true>(a, stream) : dispatch<__bf16, false>(a, stream);
    return w_transposed ? dispatch<float, true>(a, stream) : dispatch<float, false>(a, stream);
}

}  // namespace zs
