// Weight gradients of the grouped products, gfx950:
// grad_w[g] = sum over the rows i of group g of x[i]^T grad_y[i].
//
// The summed index is the row, so both operands lie in LDS in sum form and are
// read transposed.  A workgroup forms a BK x BN tile of one piece (at most
// `piece` rows) of one group.  A group of one piece is written at once; the
// pieces of a longer one leave fp32 partial sums that a second kernel adds in
// order.
#include "zs_block_internal.h"
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
};

__device__ inline int64_t clamp_offset(const int32_t* offsets, int64_t v, int64_t n_rows) {
    const int64_t o = offsets[v];
    return o < 0 ? 0 : (o > n_rows ? n_rows : o);
}

template <typename T, int BA, int BN, int WA, int WN, bool AV, bool BV>
__global__ __launch_bounds__(WA * WN * 64) void zs_wgrad_kernel(const WgParams<T> p) {
    constexpr int kWaves = WA * WN;
    constexpr int E = 16 / sizeof(T);
    constexpr int BR = kStageBytes / sizeof(T);    // rows of a stage
    constexpr int kABytes = BA * kStageBytes, kBBytes = BN * kStageBytes;
    constexpr int IA = BA / 8 / kWaves, IB = BN / 8 / kWaves;
    constexpr int AT = BA / WA / 16, NT = BN / WN / 16;
    static_assert(IA >= 1 && IB >= 1 && AT >= 1 && NT >= 1, "tile too small for its wavefronts");
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t item = xcd_item(blockIdx.x, gridDim.x);
    const int tiles = p.k_tiles * p.n_tiles;
    const int64_t slot = item / tiles;
    const int in_slot = int(item - slot * tiles);
    const int a0 = in_slot / p.n_tiles * BA, n0 = in_slot % p.n_tiles * BN;
    const auto start = [&](int64_t v) { return clamp_offset(p.offsets, v, p.n_rows); };
    const TileOf tile = find_tile(slot, p.n_groups, p.piece, start);
    if (tile.group < 0) return;
    if (tile.index > 0 && tile.begin >= tile.end) return;
    const int group = __builtin_amdgcn_readfirstlane(tile.group);

    f32x4 acc[AT][NT];
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    const int wa = wave / WN, wn = wave % WN;

    // this lane's chunks of a stage: row within the stage, first kept index
    constexpr int kALanes = BA * int(sizeof(T)) / 16, kBLanes = BN * int(sizeof(T)) / 16;
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
        bc[i] = n0 + ((chunk % kBLanes) ^ sum_swizzle<T, BN>(br[i])) * E;
    }
    const auto row_of = [&](int64_t pos) -> int64_t {
        if (pos >= tile.end) return -1;
        if (!p.perm) return pos;
        const int64_t r = p.perm[pos];
        return r >= 0 && r < p.n_rows ? r : -1;
    };
    const auto load = [&](int64_t pos, char* buf) {
#pragma unroll
        for (int i = 0; i < IA; ++i) {
            char* to = buf + (wave * IA + i) * 1024;
            const int64_t r = row_of(pos + ar[i]);
            const bool in = r >= 0 && ac[i] < p.k;
            const T* src = p.x + r * p.ldx + ac[i];
            if constexpr (AV)
                load_to_lds(in ? static_cast<const void*>(src) : zero_chunk, lds_offset(to));
            else
                *reinterpret_cast<u32x4*>(to + lane * 16) = load_partial(src, in ? p.k - ac[i] : 0);
        }
#pragma unroll
        for (int i = 0; i < IB; ++i) {
            char* to = buf + kABytes + (wave * IB + i) * 1024;
            const int64_t r = row_of(pos + br[i]);
            const bool in = r >= 0 && bc[i] < p.n;
            const T* src = p.gy + r * p.ldg + bc[i];
            if constexpr (BV)
                load_to_lds(in ? static_cast<const void*>(src) : zero_chunk, lds_offset(to));
            else
                *reinterpret_cast<u32x4*>(to + lane * 16) = load_partial(src, in ? p.n - bc[i] : 0);
        }
    };
    if (tile.begin < tile.end) {
        load(tile.begin, lds);
        wait_loads();
        __syncthreads();
        int cur = 0;
        for (int64_t pos = tile.begin; pos < tile.end; pos += BR) {
            const char* at = lds + cur * (kABytes + kBBytes);
            cur ^= 1;
            if (pos + BR < tile.end) load(pos + BR, lds + cur * (kABytes + kBBytes));
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                typename Frag<T>::V a[AT], b[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    b[j] = read_sum_frag<T, BN>(at + kABytes, wn * NT + j, s, lane);
#pragma unroll
                for (int i = 0; i < AT; ++i)
                    a[i] = read_sum_frag<T, BA>(at, wa * AT + i, s, lane);
#pragma unroll
                for (int i = 0; i < AT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[i][j] = mma16(b[j], a[i], acc[i][j]);
            }
            wait_loads();
            __syncthreads();
        }
    }

    const bool whole = tile.tiles <= 1;   // the group's only piece
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
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (n + q >= p.n) continue;
                if (whole)
                    out[at + q] = T(acc[i][j][q]);
                else
                    part[at + q] = acc[i][j][q];
            }
        }
    }
}

// Adds the partial sums of groups that were cut, in piece order.
template <typename T>
__global__ __launch_bounds__(256) void zs_wgrad_sum_kernel(const WgParams<T> p) {
    const int64_t kn = int64_t(p.k) * p.n;
    const int64_t g = blockIdx.y;
    const int64_t a = clamp_offset(p.offsets, g, p.n_rows),
                  b = clamp_offset(p.offsets, g + 1, p.n_rows);
    if (b - a <= p.piece) return;
    const int64_t pieces = (b - a + p.piece - 1) / p.piece;
    const float* from = p.partial + (a / p.piece + g) * kn;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < kn; i += int64_t(gridDim.x) * 256) {
        float s = 0.0f;
        for (int64_t j = 0; j < pieces; ++j) s += from[j * kn + i];
        p.gw[g * kn + i] = T(s);
    }
}

constexpr int kBA = 128, kBN = 128;

template <typename T>
hipError_t dispatch(const WgradArgs& a, hipStream_t stream) {
    constexpr int E = 16 / sizeof(T);
    const auto on16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    WgParams<T> p{static_cast<const T*>(a.x), static_cast<const T*>(a.gy), static_cast<T*>(a.gw),
                  a.partial, a.offsets, a.perm, a.ldx, a.ldg, a.n_rows, a.n_groups, a.piece,
                  a.k, a.n, (a.k + kBA - 1) / kBA, (a.n + kBN - 1) / kBN};
    const bool av = on16(a.x) && a.ldx % E == 0 && a.k % E == 0;
    const bool bv = on16(a.gy) && a.ldg % E == 0 && a.n % E == 0;
    const int64_t slots = a.n_rows / a.piece + a.n_groups;
    const int64_t grid = slots * p.k_tiles * p.n_tiles;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    constexpr int bytes = 2 * (kBA + kBN) * kStageBytes;
    const dim3 g{unsigned(grid)};
    if (av && bv)
        zs_wgrad_kernel<T, kBA, kBN, 2, 2, true, true><<<g, 256, bytes, stream>>>(p);
    else if (av)
        zs_wgrad_kernel<T, kBA, kBN, 2, 2, true, false><<<g, 256, bytes, stream>>>(p);
    else if (bv)
        zs_wgrad_kernel<T, kBA, kBN, 2, 2, false, true><<<g, 256, bytes, stream>>>(p);
    else
        zs_wgrad_kernel<T, kBA, kBN, 2, 2, false, false><<<g, 256, bytes, stream>>>(p);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.piece > a.n_rows) return err;
    const int64_t kn = int64_t(a.k) * a.n;
    const int64_t bx = (kn + 255) / 256;
    for (int64_t g0 = 0; g0 < a.n_groups; g0 += 65535) {   // grid.y limit
        WgParams<T> q = p;
        q.offsets += g0;
        q.gw += g0 * kn;
        q.partial += g0 * kn;
        const int64_t ng = a.n_groups - g0 < 65535 ? a.n_groups - g0 : 65535;
        zs_wgrad_sum_kernel<T><<<dim3(unsigned(bx < 4096 ? bx : 4096), unsigned(ng)), 256, 0, stream>>>(q);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

WgradPlan plan_wgrad(int64_t n_rows, int64_t n_groups, int64_t k, int64_t n, bool bf16) {
    const int64_t tiles = ((k + kBA - 1) / kBA) * ((n + kBN - 1) / kBN);
    const int64_t step = bf16 ? 64 : 32;
    constexpr int64_t kWant = 1024, kLeast = 256;
    // enough groups and tiles to fill the GPU: no group is cut
    if (n_groups * tiles >= kWant || n_rows <= kLeast) return WgradPlan{n_rows + 1, 0};
    int64_t piece = (n_rows * tiles / kWant + step - 1) / step * step;
    if (piece < kLeast) piece = kLeast;
    if (piece > n_rows) return WgradPlan{n_rows + 1, 0};
    const int64_t slots = n_rows / piece + n_groups;
    return WgradPlan{piece, size_t(slots * k * n * 4)};
}

hipError_t launch_wgrad(const WgradArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, stream) : dispatch<float>(a, stream);
}

}  // namespace zs
