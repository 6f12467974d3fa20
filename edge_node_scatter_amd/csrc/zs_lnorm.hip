// Layer norm and its gradients, gfx950.
//
//   mu = mean x, r = (mean (x - mu)^2 + eps)^(-1/2), xh = (x - mu) r, y = xh w + b
//   t = dy w,  dx = r (t - mean t - xh mean(t xh)),  dw = sum dy xh,  db = sum dy
//
// One pass over memory: a row stays in the registers of L lanes, which hold its
// 16-byte chunks l, l + L, ...; its sums cross the lanes (and, above a wavefront,
// LDS).  The mean comes first, then the sums of what is left after it and of its
// squares; the former corrects the mean, so that a row whose mean is far above its
// spread keeps its digits.  The backward pass recomputes the statistics from x; the weights' gradients are summed over a
// workgroup's rows in registers, then over its row slots in LDS, and the
// workgroups' partial sums are added in order by a second kernel.
#include "zs_layers_internal.h"
#include "zs_row.h"

namespace zs {

namespace {

template <typename T>
struct NormParams {
    const T* x;
    const float *w, *b;
    int64_t ldx, n_rows;
    int c;
    float eps, inv_c;
    bool vec;
    T* y;
    const T* gy;
    int64_t ldg;
    T* gx;
    float *gw, *gb, *partial;
};

constexpr int threads_of(int L) { return L > 256 ? L : 256; }

// x - mean in place (zeros in the places behind the row's end) and the row's
// factor r, from a row of c channels.
template <typename T, int L, int NV>
__device__ inline float centre(float (&x)[NV][Chunk<T>::V], int l, int c, float inv_c, float eps,
                               float* lds, int& region) {
    constexpr int V = Chunk<T>::V;
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += x[j][i];
    row_sum<L>(s, lds, region);
    const float mean = s[0] * inv_c;
    float d[2] = {0.0f, 0.0f};   // x - mean and its square
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[j][i] = (l + j * L) * V + i < c ? x[j][i] - mean : 0.0f;
            d[0] += x[j][i];
            d[1] = __builtin_fmaf(x[j][i], x[j][i], d[1]);
        }
    row_sum<L>(d, lds, region);
    const float rest = d[0] * inv_c;   // what the sum's roundings left in the mean
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) x[j][i] = (l + j * L) * V + i < c ? x[j][i] - rest : 0.0f;
    return 1.0f / sqrtf(__builtin_fmaf(d[1], inv_c, eps - rest * rest));
}

template <typename T, int L, int NV>
__global__ __launch_bounds__(threads_of(L)) void zs_lnorm_kernel(const NormParams<T> p) {
    constexpr int V = Chunk<T>::V;
    constexpr int kRowsOf = threads_of(L) / L;
    __shared__ float lds[2 * (L > 64 ? L / 64 : 1) * 2];
    int region = 0;
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    for (int64_t base = int64_t(blockIdx.x) * kRowsOf; base < p.n_rows;
         base += int64_t(gridDim.x) * kRowsOf) {
        const int64_t row = base + slot;
        const bool live = row < p.n_rows;
        const int c = live ? p.c : 0;
        float x[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            Chunk<T>::unpack(load_chunk(p.x + row * p.ldx, l + j * L, c, p.vec), x[j]);
        const float r = centre<T, L, NV>(x, l, c, p.inv_c, p.eps, lds, region);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = l + j * L;
            float w[V], b[V];
            load_param<V>(p.w, at, c, p.vec, w);
            if (p.b) load_param<V>(p.b, at, c, p.vec, b);
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __builtin_fmaf(x[j][i] * r, w[i], p.b ? b[i] : 0.0f);
            if (live) store_any(p.y + row * p.c, at, c, p.vec, Chunk<T>::pack(w));
        }
    }
}

// Workgroups of the backward on a compute unit: as many as the registers of a
// lane's part of a row leave room for without spilling.
template <typename T, int L, int NV>
constexpr int resident() {
    constexpr int held = NV * Chunk<T>::V;
    if (L > 256) return 1;
    return held <= 8 ? 4 : (held <= 12 ? 3 : 2);
}

template <typename T, int L, int NV>
__global__ __launch_bounds__(threads_of(L), (resident<T, L, NV>())) void zs_lnorm_bwd_kernel(
    const NormParams<T> p) {
    constexpr int V = Chunk<T>::V;
    constexpr int kThreads = threads_of(L), kRowsOf = kThreads / L;
    __shared__ float lds[2 * (L > 64 ? L / 64 : 1) * 2];
    __shared__ float sums[kRowsOf > 1 ? kThreads * V : 1];
    int region = 0;
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    float acc[2][NV][V];   // w, b
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[q][j][i] = 0.0f;
    for (int64_t base = int64_t(blockIdx.x) * kRowsOf; base < p.n_rows;
         base += int64_t(gridDim.x) * kRowsOf) {
        const int64_t row = base + slot;
        const bool live = row < p.n_rows;
        const int c = live ? p.c : 0;
        float x[NV][V], g[NV][V];
        u32x4 xr[NV], gr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            xr[j] = load_chunk(p.x + row * p.ldx, l + j * L, c, p.vec);
            gr[j] = load_chunk(p.gy + row * p.ldg, l + j * L, c, p.vec);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            Chunk<T>::unpack(xr[j], x[j]);
            Chunk<T>::unpack(gr[j], g[j]);
        }
        const float r = centre<T, L, NV>(x, l, c, p.inv_c, p.eps, lds, region);
        float s[2] = {0.0f, 0.0f};   // t, t xh
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float w[V];
            load_param<V>(p.w, l + j * L, c, p.vec, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[j][i] *= r;
                acc[0][j][i] = __builtin_fmaf(g[j][i], x[j][i], acc[0][j][i]);
                acc[1][j][i] += g[j][i];
                g[j][i] *= w[i];
                s[0] += g[j][i];
                s[1] = __builtin_fmaf(g[j][i], x[j][i], s[1]);
            }
        }
        row_sum<L>(s, lds, region);
        const float mt = s[0] * p.inv_c, mx = s[1] * p.inv_c;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) g[j][i] = r * (g[j][i] - mt - x[j][i] * mx);
            if (live) store_any(p.gx + row * p.c, l + j * L, c, p.vec, Chunk<T>::pack(g[j]));
        }
    }
    // sums over the workgroup's row slots, then out: [2][c] per workgroup
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float* out = p.partial + (int64_t(blockIdx.x) * 2 + q) * p.c;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (kRowsOf > 1) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < V; ++i) sums[(slot * L + l) * V + i] = acc[q][j][i];
                __syncthreads();
                for (int e = threadIdx.x; e < L * V; e += kThreads) {
                    const int ch = j * L * V + e;
                    float s = 0.0f;
                    for (int k = 0; k < kRowsOf; ++k) s += sums[k * L * V + e];
                    if (ch < p.c) out[ch] = s;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int ch = (j * L + l) * V + i;
                    if (ch < p.c) out[ch] = acc[q][j][i];
                }
            }
        }
    }
}

// Adds the workgroups' partial sums in order: 32 columns a workgroup, 32 lanes of
// partial rows each, joined in LDS.
__global__ __launch_bounds__(1024) void zs_lnorm_sum_kernel(const float* partial, int count, int c,
                                                            float* gw, float* gb) {
    __shared__ float lds[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    float s = 0.0f;
    if (col < 2 * c) {
#pragma unroll 4
        for (int i = part; i < count; i += 32) s += partial[int64_t(i) * 2 * c + col];
    }
    lds[part][threadIdx.x & 31] = s;
    __syncthreads();
    if (part == 0 && col < 2 * c) {
        s = 0.0f;
        for (int i = 0; i < 32; ++i) s += lds[i][threadIdx.x];
        float* out = col < c ? gw : gb;
        if (out) out[col % c] = s;
    }
}

constexpr int64_t kMaxPartials = 1024;

template <typename T, int L, int NV>
hipError_t run(const NormArgs& a, bool backward, hipStream_t stream) {
    constexpr int V = Chunk<T>::V, rows = threads_of(L) / L;
    const auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    NormParams<T> p{};
    p.x = static_cast<const T*>(a.x), p.w = a.w, p.b = a.b;
    p.ldx = a.ldx, p.n_rows = a.n_rows, p.c = a.c, p.eps = a.eps, p.inv_c = 1.0f / float(a.c);
    p.y = static_cast<T*>(a.y);
    p.gy = static_cast<const T*>(a.gy), p.ldg = a.ldg, p.gx = static_cast<T*>(a.gx);
    p.gw = a.gw, p.gb = a.gb, p.partial = a.partial;
    p.vec = a.c % V == 0 && a.ldx % V == 0 && on16(a.x) && on16(a.y) && on16(a.w) && on16(a.b) &&
            a.ldg % V == 0 && on16(a.gy) && on16(a.gx);
    const int64_t want = (p.n_rows + rows - 1) / rows;
    if (!backward) {
        zs_lnorm_kernel<T, L, NV>
            <<<unsigned(want < 8192 ? want : 8192), threads_of(L), 0, stream>>>(p);
        return hipGetLastError();
    }
    // one round of workgroups that all run at once
    constexpr int64_t cap = 256 * resident<T, L, NV>();
    static_assert(cap <= kMaxPartials, "partial sums for every workgroup");
    const unsigned grid = unsigned(want < cap ? want : cap);
    if (grid > 0) {
        zs_lnorm_bwd_kernel<T, L, NV><<<grid, threads_of(L), 0, stream>>>(p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    zs_lnorm_sum_kernel<<<(2 * p.c + 31) / 32, 1024, 0, stream>>>(p.partial, int(grid), p.c, p.gw,
                                                                  p.gb);
    return hipGetLastError();
}

// Lanes and chunks per lane by the row's width in chunks: the fewest lanes that
// hold a row in one chunk each up to a wavefront, then two or three chunks a lane,
// then a workgroup.
template <typename T>
hipError_t dispatch(const NormArgs& a, bool backward, hipStream_t stream) {
    const int chunks = (a.c + Chunk<T>::V - 1) / Chunk<T>::V;
    if (chunks <= 1) return run<T, 1, 1>(a, backward, stream);
    if (chunks <= 2) return run<T, 2, 1>(a, backward, stream);
    if (chunks <= 4) return run<T, 4, 1>(a, backward, stream);
    if (chunks <= 8) return run<T, 8, 1>(a, backward, stream);
    if (chunks <= 16) return run<T, 16, 1>(a, backward, stream);
    if (chunks <= 32) return run<T, 32, 1>(a, backward, stream);
    if (chunks <= 64) return run<T, 64, 1>(a, backward, stream);
    if (chunks <= 128) return run<T, 64, 2>(a, backward, stream);
    if (chunks <= 192) return run<T, 64, 3>(a, backward, stream);
    if (chunks <= 256) return run<T, 256, 1>(a, backward, stream);
    if (chunks <= 512) return run<T, 256, 2>(a, backward, stream);
    if constexpr (sizeof(T) == 2) return run<T, 512, 2>(a, backward, stream);
    if (chunks <= 1024) return run<T, 256, 4>(a, backward, stream);
    return run<T, 512, 4>(a, backward, stream);
}

}  // namespace

size_t layer_norm_workspace(int64_t n_rows, int64_t c) {
    const int64_t parts = n_rows < kMaxPartials ? n_rows : kMaxPartials;
    return size_t(parts * 2 * c * 4);
}

hipError_t launch_layer_norm(const NormArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, false, stream) : dispatch<float>(a, false, stream);
}

hipError_t launch_layer_norm_backward(const NormArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, true, stream) : dispatch<float>(a, true, stream);
}

}  // namespace zs
