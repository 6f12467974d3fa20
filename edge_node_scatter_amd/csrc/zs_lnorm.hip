// Layer norm and its gradients, gfx950.
//
//   mu = mean x, r = (mean (x - mu)^2 + eps)^(-1/2), xh = (x - mu) r, y = xh w + b
//   t = dy w,  dx = r (t - mean t - xh mean(t xh)),  dw = sum dy xh,  db = sum dy
//
// One pass over memory: a row stays in the registers of L lanes, which hold its
// 16-byte chunks l, l + L, ...; its sums cross the lanes (and, above a wavefront,
// LDS).  The mean comes first, then the sums of what is left after it and of its
// squares; the former corrects the mean, so that a row whose mean is far above its
// spread keeps its digits.  Where the mean's rounding is most of what is left (equal
// elements far from zero) it is taken off once more: without that step 892 times 7.3e9 gave
// 0.03 for 0, and gradients whose factor was that of the rounding, not of eps.
// The backward pass recomputes the statistics from x; the weights' gradients are summed
// over a workgroup's rows in registers, then over its row slots in LDS, and the
// workgroups' partial sums are added in order by a second kernel.
//
// Bound by memory.  Measured on MI355X (a copy reaches 5.15 TB/s):
//  - gradients of 32768 x 2048 in bf16: 72 us and 5 us for the partial sums, 5.6
//    TB/s of 403 MB.  A wavefront a row, four chunks a lane, no barrier, the next
//    row's loads in flight; 88 us with a workgroup a row, 120 without the loads ahead,
//    94 with w read from memory and the deviations formed anew in each pass.
//  - gradients of 4096 x 8192 in fp32: call 79 us, 5.1 TB/s of 403 MB; 97 where lanes behind
//    the row's end skipped their loads (8192 x 8192 in bf16 92, 95 so).
//  - forward of 8191 x 777 in fp32: 12 us, 4.1 TB/s of 51 MB: no row starts on 16 bytes
//    (23 us with parameters and results channel by channel).
#include <climits>

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
    bool stream;   // the gradient goes past the caches
    T* y;
    const T* gy;
    int64_t ldg;
    T* gx;
    float *gw, *gb, *partial;
};

constexpr int threads_of(int L) { return L > 256 ? L : 256; }

// Rows on 16 bytes of whole chunks (WHOLE) have code without tests of single
// channels; the others test each in the row's last chunk.
template <typename T, bool WHOLE>
__device__ inline u32x4 load_x(const T* row, int chunk, int c) {
    return load_raw<T, true>(row, chunk, c, WHOLE);
}
// Calls f(i, whether channel i of the chunk is the row's) for the chunk's channels, if
// the chunk has any.
template <int V, bool WHOLE, typename F>
__device__ inline void each(int chunk, int c, F f) {
    const int left = c - chunk * V;
    if (left <= 0) return;
#pragma unroll
    for (int i = 0; i < V; ++i) f(i, WHOLE || i < left);
}
// V fp32 parameters of a chunk that starts anywhere.
template <int V, bool WHOLE>
__device__ inline void load_weights(const float* p, int chunk, int c, float (&f)[V]) {
    if (WHOLE || c - chunk * V >= V) {
        __builtin_memcpy(f, __builtin_assume_aligned(p + chunk * V, WHOLE ? 16 : 4), sizeof f);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = chunk * V + i < c ? p[chunk * V + i] : 0.0f;
    }
}

// What turns a row's deviations d = x - mean into its normalised values d r + shift:
// the factor, and minus the factor times what the first sum's roundings left of the
// mean.  d is small where the row's mean is far above its spread, so nothing is lost.
struct Stats {
    float r, shift;
};
template <typename T, int L, int NV, bool WHOLE>
__device__ inline Stats deviations(const u32x4 (&raw)[NV], float (&d)[NV][Chunk<T>::V], int l,
                                   int c, float inv_c, float eps, float* lds, int& region) {
    constexpr int V = Chunk<T>::V;
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        // zeros behind the row's end
        Chunk<T>::unpack(settled<T>(raw[j], l + j * L, c, WHOLE), d[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += d[j][i];
    }
    row_sum<L>(s, lds, region);
    const float mean = s[0] * inv_c;
    float q[2] = {0.0f, 0.0f};   // d and its square
#pragma unroll
    for (int j = 0; j < NV; ++j)
        each<V, WHOLE>(l + j * L, c, [&](int i, bool in) {
            d[j][i] = in ? d[j][i] - mean : 0.0f;
            q[0] += d[j][i];
            q[1] = __builtin_fmaf(d[j][i], d[j][i], q[1]);
        });
    row_sum<L>(q, lds, region);
    float rest = q[0] * inv_c, square = q[1] * inv_c;
    // Where the mean's rounding is most of the deviations, the variance below is a difference
    // without digits: rest is taken off them, as often as it takes.  Once is enough for any
    // spread; what rounding leaves of equal elements gets 2^-20 or so smaller at a time and
    // ends when it is nothing against eps.  (Squares of 1e19 are inf, on both sides here.)
    for (int step = 0; step < 16; ++step) {   // of all the row's lanes alike
        const bool again = rest * q[0] >= 0.5f * __builtin_fminf(q[1], __FLT_MAX__) &&
                           square > eps * 0x1p-16f;
        if (__ballot(again) == 0) break;
        const float off = again ? rest : 0.0f;
        q[0] = q[1] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            each<V, WHOLE>(l + j * L, c, [&](int i, bool in) {
                d[j][i] = in ? d[j][i] - off : 0.0f;
                q[0] += d[j][i];
                q[1] = __builtin_fmaf(d[j][i], d[j][i], q[1]);
            });
        row_sum<L>(q, lds, region);
        rest = q[0] * inv_c, square = q[1] * inv_c;
    }
    Stats t;
    // (the difference of two rounded values can be below 0 where all deviations are the same)
    const float var = __builtin_fmaf(-rest, rest, square);
    t.r = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);
    t.shift = -rest * t.r;
    return t;
}

template <typename T, int L, int NV, bool WHOLE>
__global__ __launch_bounds__(threads_of(L)) void zs_lnorm_kernel(const NormParams<T> p) {
    constexpr int V = Chunk<T>::V;
    constexpr int kRowsOf = threads_of(L) / L;
    __shared__ float lds[2 * (L > 64 ? L / 64 : 1) * 2];
    int region = 0;
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    for (int64_t base = int64_t(blockIdx.x) * kRowsOf; base < p.n_rows;
         base += int64_t(gridDim.x) * kRowsOf) {
        const int64_t row = base + slot;
        const int c = row < p.n_rows ? p.c : 0;
        u32x4 raw[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) raw[j] = load_x<T, WHOLE>(p.x + row * p.ldx, l + j * L, c);
        float d[NV][V];
        const Stats t = deviations<T, L, NV, WHOLE>(raw, d, l, c, p.inv_c, p.eps, lds, region);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = l + j * L;
            if (at * V >= c) continue;
            float w[V], b[V];
            load_weights<V, WHOLE>(p.w, at, c, w);
            if (p.b) load_weights<V, WHOLE>(p.b, at, c, b);
#pragma unroll
            for (int i = 0; i < V; ++i)
                d[j][i] = __builtin_fmaf(__builtin_fmaf(d[j][i], t.r, t.shift), w[i],
                                         p.b ? b[i] : 0.0f);
            store_any(p.y + row * p.c, at, c, WHOLE, Chunk<T>::pack(d[j]));
        }
    }
}

// Wavefronts of the backward on a SIMD: as many as the registers of a lane's part of a
// row (its values, both sums, and both inputs of this row and the next as they lie in
// memory) leave room for without spilling.  Rows of 512 lanes take whole workgroups
// of two wavefronts a SIMD: two of them where they fit (8192 x 8192 in bf16 95 us then, 112
// with one; in fp32 two would spill, 104 us against 92).
template <typename T, int L, int NV>
constexpr int resident() {
    constexpr int held = NV * (3 * Chunk<T>::V + 16);
    if (L > 256) return held <= 80 ? 4 : 2;
    return held <= 56 ? 4 : (held <= 120 ? 3 : 2);
}

// Chunk `chunk` of a row, which has it.  (A row of less than a chunk is one lane's.)
template <typename T, int L, bool WHOLE>
__device__ inline u32x4 load_inside(const T* row, int chunk, int c) {
    constexpr int V = Chunk<T>::V;
    if constexpr (WHOLE) return load_chunk<T, true>(row, chunk, INT_MAX, true);
    if constexpr (L == 1) return load_raw(row, chunk, c, false);
    const int at = chunk * V < c - V ? chunk * V : c - V;
    u32x4 v;
    __builtin_memcpy(&v, row + at, 16);
    return v;
}

// A lane's part of a row's inputs as they lie in memory, read once and past the
// caches.  Lanes behind the row's end load its last chunk and rows behind the last one the
// last: where loads may be skipped, nobody can count them, and a wait for this row's is one
// for the next row's too.
template <int NV>
struct RowInputs {
    u32x4 x[NV], gy[NV];
};
template <typename T, int L, int NV, bool WHOLE>
__device__ inline RowInputs<NV> load_row(const NormParams<T>& p, int64_t row, int l) {
    RowInputs<NV> r;
    const int64_t at = row < p.n_rows ? row : p.n_rows - 1;
    const int last = (p.c - 1) / Chunk<T>::V;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int chunk = l + j * L < last ? l + j * L : last;
        r.x[j] = load_inside<T, L, WHOLE>(p.x + at * p.ldx, chunk, p.c);
        r.gy[j] = load_inside<T, L, WHOLE>(p.gy + at * p.ldg, chunk, p.c);
    }
    return r;
}

template <typename T, int L, int NV, bool WHOLE>
__global__ __launch_bounds__(threads_of(L), (resident<T, L, NV>())) void zs_lnorm_bwd_kernel(
    const NormParams<T> p) {
    constexpr int V = Chunk<T>::V;
    constexpr int kThreads = threads_of(L), kRowsOf = kThreads / L;
    __shared__ float lds[2 * (L > 64 ? L / 64 : 1) * 2];
    // w, four channels of every chunk at a time, so that the lanes' reads are
    // contiguous.  In LDS because loads return in order: a wait for w from memory
    // would wait for the next row too.
    __shared__ __align__(16) float weights[V / 4][NV * L][4];
    __shared__ float sums[kRowsOf > 1 ? kThreads * V : 1];
    int region = 0;
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    for (int ch = threadIdx.x; ch < NV * L * V; ch += kThreads)
        weights[ch % V / 4][ch / V][ch % 4] = ch < p.c ? p.w[ch] : 0.0f;
    __syncthreads();
    const auto weight_of = [&](int at, float (&w)[V]) {
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            const f32x4 t = *reinterpret_cast<const f32x4*>(weights[h][at]);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[h * 4 + i] = t[i];
        }
    };
    float acc[2][NV][V];   // w, b
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[q][j][i] = 0.0f;
    // the next row's loads are in flight while this one is used
    const int64_t step = int64_t(gridDim.x) * kRowsOf;
    RowInputs<NV> next = load_row<T, L, NV, WHOLE>(p, int64_t(blockIdx.x) * kRowsOf + slot, l);
    for (int64_t base = int64_t(blockIdx.x) * kRowsOf; base < p.n_rows; base += step) {
        const int64_t row = base + slot;
        const int c = row < p.n_rows ? p.c : 0;
        const RowInputs<NV> in = next;
        next = load_row<T, L, NV, WHOLE>(p, row + step, l);
        float x[NV][V];
        u32x4 raw[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            raw[j] = !WHOLE || (l + j * L) * V < c ? in.x[j] : u32x4{0, 0, 0, 0};
        const Stats t = deviations<T, L, NV, WHOLE>(raw, x, l, c, p.inv_c, p.eps, lds, region);
        float s[2] = {0.0f, 0.0f};   // t, t xh
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = l + j * L;
            if (at * V >= c) continue;
            float g[V], w[V];
            Chunk<T>::unpack(settled<T>(in.gy[j], at, c, WHOLE), g);
            weight_of(at, w);
            // behind the row's end g and w are zeros
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[j][i] = __builtin_fmaf(x[j][i], t.r, t.shift);
                acc[0][j][i] = __builtin_fmaf(g[i], x[j][i], acc[0][j][i]);
                acc[1][j][i] += g[i];
                const float u = g[i] * w[i];
                s[0] += u;
                s[1] = __builtin_fmaf(u, x[j][i], s[1]);
            }
        }
        row_sum<L>(s, lds, region);
        const float mt = s[0] * p.inv_c, mx = s[1] * p.inv_c;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = l + j * L;
            if (at * V >= c) continue;
            float g[V], w[V];
            Chunk<T>::unpack(settled<T>(in.gy[j], at, c, WHOLE), g);
            weight_of(at, w);
#pragma unroll
            for (int i = 0; i < V; ++i)
                g[i] = t.r * __builtin_fmaf(-mx, x[j][i], __builtin_fmaf(g[i], w[i], -mt));
            if (WHOLE)
                store_chunk(p.gx + row * p.c, at, c, true, Chunk<T>::pack(g), p.stream);
            else
                store_any(p.gx + row * p.c, at, c, false, Chunk<T>::pack(g));
        }
    }
    // sums over the workgroup's row slots, then out: [2][c] per workgroup.  A single
    // workgroup's are the gradients.
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float* out = p.partial + (int64_t(blockIdx.x) * 2 + q) * p.c;
        if (gridDim.x == 1) out = q == 0 ? p.gw : p.gb;
        if (!out) continue;
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

template <typename T, int L, int NV, bool WHOLE>
hipError_t run_kernels(const NormParams<T>& p, bool backward, hipStream_t stream) {
    constexpr int rows = threads_of(L) / L;
    const int64_t want = (p.n_rows + rows - 1) / rows;
    if (!backward) {
        zs_lnorm_kernel<T, L, NV, WHOLE>
            <<<unsigned(want < 8192 ? want : 8192), threads_of(L), 0, stream>>>(p);
        return hipGetLastError();
    }
    // one round of workgroups that all run at once
    constexpr int64_t cap = 256 * resident<T, L, NV>() * 256 / threads_of(L);
    static_assert(cap <= kMaxPartials, "partial sums for every workgroup");
    const unsigned grid = unsigned(want < cap ? want : cap);
    if (grid > 0) {
        zs_lnorm_bwd_kernel<T, L, NV, WHOLE><<<grid, threads_of(L), 0, stream>>>(p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess || grid == 1) return err;
    }
    zs_lnorm_sum_kernel<<<(2 * p.c + 31) / 32, 1024, 0, stream>>>(p.partial, int(grid), p.c, p.gw,
                                                                  p.gb);
    return hipGetLastError();
}

template <typename T, int L, int NV>
hipError_t run(const NormArgs& a, bool backward, hipStream_t stream) {
    constexpr int V = Chunk<T>::V;
    const auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    NormParams<T> p{};
    p.x = static_cast<const T*>(a.x), p.w = a.w, p.b = a.b;
    p.ldx = a.ldx, p.n_rows = a.n_rows, p.c = a.c, p.eps = a.eps, p.inv_c = 1.0f / float(a.c);
    p.y = static_cast<T*>(a.y);
    p.gy = static_cast<const T*>(a.gy), p.ldg = a.ldg, p.gx = static_cast<T*>(a.gx);
    p.gw = a.gw, p.gb = a.gb, p.partial = a.partial;
    // as in the join's backward: outputs that fill half of the memory-side cache alone
    p.stream = a.n_rows * a.c * int64_t(sizeof(T)) >= (int64_t(128) << 20);
    const bool whole = a.c % V == 0 && a.ldx % V == 0 && on16(a.x) && on16(a.y) && on16(a.w) &&
                       on16(a.b) && a.ldg % V == 0 && on16(a.gy) && on16(a.gx);
    return whole ? run_kernels<T, L, NV, true>(p, backward, stream)
                 : run_kernels<T, L, NV, false>(p, backward, stream);
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
    if (chunks <= 256) return run<T, 64, 4>(a, backward, stream);
    if constexpr (sizeof(T) == 2) {
        if (chunks <= 512) return run<T, 256, 2>(a, backward, stream);
        return run<T, 512, 2>(a, backward, stream);
    } else {
        if (chunks <= 512) return run<T, 256, 2>(a, backward, stream);
        if (chunks <= 1024) return run<T, 256, 4>(a, backward, stream);
        return run<T, 512, 4>(a, backward, stream);
    }
}

}  // namespace

// Nothing where one workgroup holds all rows, whose sums are the gradients (a row's
// lanes in fp32: in bf16 there are no more).
size_t layer_norm_workspace(int64_t n_rows, int64_t c) {
    int lanes = 1;
    while (lanes < 64 && lanes * 4 < c) lanes *= 2;
    if (n_rows <= (c <= 1024 ? 256 / lanes : 1)) return 0;
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
