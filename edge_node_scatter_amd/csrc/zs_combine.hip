// Weighted sum of the experts' rows of a token and its gradients, gfx950.
//
//   y[t] = sum_j w[t][j] z[t k + j];  dz[t k + j] = w[t][j] dy[t],
//   dw[t][j] = <dy[t], z[t k + j]>
//
// Bound by memory: every row of z is read once.  Forward: a lane holds a chunk of y
// and takes its slots four loads at a time.  Backward: the L lanes of a token hold
// dy[t], so that it is read once too, and the k dot products cross the lanes (and,
// above a wavefront, LDS).
#include "zs_launch.h"
#include "zs_layers_internal.h"
#include "zs_row.h"

namespace zs {

namespace {

constexpr int kThreads = 256;

template <typename T>
struct CombineParams {
    const T* z;
    const float* weight;
    int64_t ldz, n_rows, block0;
    int k, c, blocks;   // column blocks of L chunks
    bool vec;
    bool stream;   // the backward's gradient goes past the caches
    T* y;
    const T* gy;
    int64_t ldg;
    T* gz;
    float* gw;
};

// WHOLE: rows on 16 bytes of whole chunks.
template <typename T, int L, bool WHOLE>
__global__ __launch_bounds__(kThreads) void zs_combine_kernel(const CombineParams<T> p) {
    constexpr int V = Chunk<T>::V, kRows = kThreads / L, kLoads = 4;
    const int64_t block = p.block0 + blockIdx.x;
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    const int64_t t = block / p.blocks * kRows + slot;
    const int chunk = int(block % p.blocks) * L + l;
    if (t >= p.n_rows || chunk * V >= p.c) return;
    const T* z = p.z + t * p.k * p.ldz;
    const float* w = p.weight + t * p.k;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    const auto add = [&](int j, u32x4 raw) {
        float f[V];
        Chunk<T>::unpack(settled<T>(raw, chunk, p.c, WHOLE), f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w[j], f[i], acc[i]);
    };
    int j = 0;
    for (; j + kLoads <= p.k; j += kLoads) {
        u32x4 raw[kLoads];
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
            raw[q] = load_raw(z + (j + q) * p.ldz, chunk, p.c, WHOLE);
#pragma unroll
        for (int q = 0; q < kLoads; ++q) add(j + q, raw[q]);
    }
    // the rest two at a time (31837 x 2 x 832 in bf16 27 us, 29 one by one)
    for (; j + 2 <= p.k; j += 2) {
        const u32x4 raw0 = load_raw(z + j * p.ldz, chunk, p.c, WHOLE);
        const u32x4 raw1 = load_raw(z + (j + 1) * p.ldz, chunk, p.c, WHOLE);
        add(j, raw0), add(j + 1, raw1);
    }
    if (j < p.k) add(j, load_raw(z + j * p.ldz, chunk, p.c, WHOLE));
    store_any(p.y + t * p.c, chunk, p.c, WHOLE, Chunk<T>::pack(acc));
}

constexpr int threads_of(int L) { return L > kThreads ? L : kThreads; }

// Rows on 16 bytes of whole chunks (WHOLE) have code without tests of single
// channels.  U slots' rows are in flight while as many are used: they are asked for
// before those results are stored, as a wait for a load waits for every store before
// it.
template <typename T, int L, int NV, bool WHOLE>
__global__ __launch_bounds__(threads_of(L)) void zs_combine_bwd_kernel(const CombineParams<T> p) {
    constexpr int V = Chunk<T>::V, kRows = threads_of(L) / L, kWaves = L > 64 ? L / 64 : 1;
    constexpr int U = NV > 2 ? 1 : 2;
    __shared__ float dots[kWaves > 1 ? kWaves * ZS_MAX_SLOTS : 1];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    for (int64_t base = int64_t(blockIdx.x) * kRows; base < p.n_rows;
         base += int64_t(gridDim.x) * kRows) {
        const int64_t t = base + slot;
        const bool live = t < p.n_rows;
        const int c = live ? p.c : 0;
        u32x4 next[U][NV];
        float next_w[U];
        const auto load = [&](int j0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = t * p.k + j0 + u;
                const bool in = live && j0 + u < p.k;
                next_w[u] = in ? p.weight[row] : 0.0f;
#pragma unroll
                for (int n = 0; n < NV; ++n)
                    next[u][n] = load_raw<T, true>(p.z + row * p.ldz, l + n * L, in ? c : 0, WHOLE);
            }
        };
        float g[NV][V];
        u32x4 raw_g[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n)
            raw_g[n] = load_raw<T, true>(p.gy + t * p.ldg, l + n * L, c, WHOLE);
        load(0);
#pragma unroll
        for (int n = 0; n < NV; ++n)
            Chunk<T>::unpack(settled<T>(raw_g[n], l + n * L, c, WHOLE), g[n]);
        if constexpr (kWaves > 1) __syncthreads();   // the last token's dots are read
        for (int j0 = 0; j0 < p.k; j0 += U) {
            u32x4 raw[U][NV];
            float w[U], dot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = next_w[u];
#pragma unroll
                for (int n = 0; n < NV; ++n) raw[u][n] = next[u][n];
            }
            load(j0 + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = t * p.k + j0 + u;
                const bool in = live && j0 + u < p.k;
                dot[u] = 0.0f;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int at = l + n * L;
                    float z[V];
                    Chunk<T>::unpack(settled<T>(raw[u][n], at, c, WHOLE), z);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dot[u] = __builtin_fmaf(g[n][i], z[i], dot[u]);
                        z[i] = w[u] * g[n][i];
                    }
                    if (!in || at * V >= c) continue;
                    if (WHOLE)
                        store_chunk(p.gz + row * p.c, at, c, true, Chunk<T>::pack(z), p.stream);
                    else
                        store_any(p.gz + row * p.c, at, c, false, Chunk<T>::pack(z));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) dot[u] = lane_sum<(L < 64 ? L : 64)>(dot[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (j0 + u >= p.k) continue;
                if constexpr (kWaves > 1) {
                    if ((threadIdx.x & 63) == 0)
                        dots[(threadIdx.x >> 6) * ZS_MAX_SLOTS + j0 + u] = dot[u];
                } else if (l == 0 && live) {
                    p.gw[t * p.k + j0 + u] = dot[u];
                }
            }
        }
        if constexpr (kWaves > 1) {
            __syncthreads();
            if (int(threadIdx.x) < p.k) {
                float s = 0.0f;
#pragma unroll
                for (int v = 0; v < kWaves; ++v) s += dots[v * ZS_MAX_SLOTS + threadIdx.x];
                p.gw[t * p.k + threadIdx.x] = s;
            }
        }
    }
}

template <typename T>
CombineParams<T> params(const CombineArgs& a) {
    constexpr int V = Chunk<T>::V;
    const auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    CombineParams<T> p{};
    p.z = static_cast<const T*>(a.z), p.weight = a.weight, p.ldz = a.ldz, p.n_rows = a.n_rows;
    p.k = a.k, p.c = a.c, p.y = static_cast<T*>(a.y);
    p.gy = static_cast<const T*>(a.gy), p.ldg = a.ldg, p.gz = static_cast<T*>(a.gz), p.gw = a.gw;
    p.vec = a.c % V == 0 && a.ldz % V == 0 && a.ldg % V == 0 && on16(a.z) && on16(a.y) &&
            on16(a.gy) && on16(a.gz);
    // as in the join's backward: outputs that fill half of the memory-side cache alone
    p.stream = a.n_rows * a.k * a.c * int64_t(sizeof(T)) >= (int64_t(128) << 20);
    return p;
}

template <typename T, int L>
hipError_t run(const CombineArgs& a, hipStream_t stream) {
    constexpr int V = Chunk<T>::V, kRows = kThreads / L;
    CombineParams<T> p = params<T>(a);
    p.blocks = ((a.c + V - 1) / V + L - 1) / L;
    const int64_t grid = (a.n_rows + kRows - 1) / kRows * p.blocks;
    return launch_ranges(grid, kThreads, [&](int64_t first, int64_t count) {
        p.block0 = first;
        if (p.vec) zs_combine_kernel<T, L, true><<<unsigned(count), kThreads, 0, stream>>>(p);
        else zs_combine_kernel<T, L, false><<<unsigned(count), kThreads, 0, stream>>>(p);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t dispatch(const CombineArgs& a, hipStream_t stream) {
    const int chunks = (a.c + Chunk<T>::V - 1) / Chunk<T>::V;
    if (chunks <= 1) return run<T, 1>(a, stream);
    if (chunks <= 2) return run<T, 2>(a, stream);
    if (chunks <= 4) return run<T, 4>(a, stream);
    if (chunks <= 8) return run<T, 8>(a, stream);
    if (chunks <= 16) return run<T, 16>(a, stream);
    if (chunks <= 32) return run<T, 32>(a, stream);
    return run<T, 64>(a, stream);
}

template <typename T, int L, int NV>
hipError_t run_bwd(const CombineArgs& a, hipStream_t stream) {
    constexpr int kRows = threads_of(L) / L;
    const CombineParams<T> p = params<T>(a);
    const int64_t want = (a.n_rows + kRows - 1) / kRows;
    const unsigned grid = unsigned(want < 8192 ? want : 8192);
    if (p.vec)
        zs_combine_bwd_kernel<T, L, NV, true><<<grid, threads_of(L), 0, stream>>>(p);
    else
        zs_combine_bwd_kernel<T, L, NV, false><<<grid, threads_of(L), 0, stream>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t dispatch_bwd(const CombineArgs& a, hipStream_t stream) {
    const int chunks = (a.c + Chunk<T>::V - 1) / Chunk<T>::V;
    if (chunks <= 1) return run_bwd<T, 1, 1>(a, stream);
    if (chunks <= 2) return run_bwd<T, 2, 1>(a, stream);
    if (chunks <= 4) return run_bwd<T, 4, 1>(a, stream);
    if (chunks <= 8) return run_bwd<T, 8, 1>(a, stream);
    if (chunks <= 16) return run_bwd<T, 16, 1>(a, stream);
    if (chunks <= 32) return run_bwd<T, 32, 1>(a, stream);
    if (chunks <= 64) return run_bwd<T, 64, 1>(a, stream);
    if (chunks <= 128) return run_bwd<T, 64, 2>(a, stream);
    if (chunks <= 256) return run_bwd<T, 64, 4>(a, stream);
    if (chunks <= 512) return run_bwd<T, 256, 2>(a, stream);
    if (chunks <= 1024) return run_bwd<T, 256, 4>(a, stream);
    return run_bwd<T, 512, 4>(a, stream);
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, stream) : dispatch<float>(a, stream);
}

hipError_t launch_combine_backward(const CombineArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch_bwd<__bf16>(a, stream) : dispatch_bwd<float>(a, stream);
}

}  // namespace zs
