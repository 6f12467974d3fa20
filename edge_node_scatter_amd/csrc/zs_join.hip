// The gated residual join between two norms and its gradients, gfx950.
//
//   u = zn w_post, zn = z rz, rz = (mean z^2 + eps)^(-1/2)
//   y = x + scale s u, s = sigmoid(gate);  h = yn w_pre, yn = y ry, ry likewise
//
// backward, with t = gh w_pre and everything recomputed from the inputs:
//   gx = gy + ry (t - yn mean(t yn))
//   b = gx s, q = b scale, r = q w_post
//   gz = rz (r - zn mean(r zn)),  ggate = q u (1 - s)
//   gscale = sum b u, gpost = sum q zn, gpre = sum gh yn   (over the rows)
//
// No power of ry or rz is formed: a cube leaves fp32's range where the row's norm is
// under 1e-13 or above 1e13, and times the zero lanes of absent rows it would be NaN.
//
// One pass over memory: a row stays in the registers of L lanes, which hold its
// 16-byte chunks l, l + L, ...; the row sums cross the lanes (and, above a
// wavefront, LDS).  The parameter gradients are summed over a workgroup's rows
// in registers, then over its row slots in LDS, and the workgroups' partial
// sums are added in order by a second kernel.
//
// Bound by memory.  Measured on MI355X (a copy reaches 5.1 TB/s):
//  - gradients of 32768 x 2048 in bf16: 241 us and 5 us for the partial sums, 4.5 TB/s
//    of 1.07 GB; some 60 vector instructions an element beside them (a workgroup a
//    row, a chunk a lane, the next row's loads in flight; without those 363 us).
//  - gradients of 16384 x 520 in fp32: 44 and 4 us, 4.7 TB/s of 205 MB (130 chunks of
//    a wavefront's 192).
//  - forward of 65536 x 32 in fp32: 9.7 us, 4.3 TB/s of 42 MB.
#include "zs_block_internal.h"
#include "zs_tile.h"

namespace zs {

namespace {

template <typename T>
struct Chunk {
    static constexpr int V = 16 / sizeof(T);
    __device__ static void unpack(u32x4 raw, float (&f)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bits = raw[i];
                f[i] = __builtin_bit_cast(float, bits);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __builtin_bit_cast(float, raw[i] << 16);
                f[2 * i + 1] = __builtin_bit_cast(float, raw[i] & 0xffff0000u);
            }
        }
    }
    __device__ static u32x4 pack(const float (&f)[V]) {
        union {
            T e[V];
            u32x4 v;
        } u;
#pragma unroll
        for (int i = 0; i < V; ++i) u.e[i] = T(f[i]);
        return u.v;
    }
};

// Chunk `chunk` of a row of c elements (zeros outside).  vec: whole chunks on 16
// bytes; NT: read once, past the caches.
template <typename T, bool NT = false>
__device__ inline u32x4 load_chunk(const T* row, int chunk, int c, bool vec) {
    constexpr int V = Chunk<T>::V;
    const int left = c - chunk * V;
    if (NT && vec)
        return left > 0
                   ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + chunk * V))
                   : u32x4{0, 0, 0, 0};
    if (vec) return left > 0 ? *reinterpret_cast<const u32x4*>(row + chunk * V) : u32x4{0, 0, 0, 0};
    return load_partial(row + chunk * V, left);
}
template <typename T>
__device__ inline void store_chunk(T* row, int chunk, int c, bool vec, u32x4 v,
                                   bool stream = false) {
    constexpr int V = Chunk<T>::V;
    const int left = c - chunk * V;
    if (vec && stream) {
        if (left > 0) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(row + chunk * V));
        return;
    }
    if (vec) {
        if (left > 0) *reinterpret_cast<u32x4*>(row + chunk * V) = v;
        return;
    }
    union {
        u32x4 v;
        T e[V];
    } u;
    u.v = v;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < left) row[chunk * V + i] = u.e[i];
}
// V fp32 parameters of a chunk.
template <int V>
__device__ inline void load_param(const float* p, int chunk, int c, bool vec, float (&f)[V]) {
    const int left = c - chunk * V;
    if (vec) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4 t = left > 0 ? *reinterpret_cast<const f32x4*>(p + chunk * V + i)
                                     : f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) f[i + q] = t[q];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i < left ? p[chunk * V + i] : 0.0f;
    }
}

// v of the lane that a DPP control picks within 16 lanes.
template <int CTRL>
__device__ inline float dpp(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// Sum over the L <= 64 lanes of a row, in all of them, without LDS: halves are
// exchanged within 16 lanes by DPP (xor 1, xor 2, mirrors of 8 and 16 lanes),
// then across 16 and 32 lanes by the permlane swaps, whose two results are the
// two halves.
template <int L>
__device__ inline float lane_sum(float v) {
    if constexpr (L >= 2) v += dpp<0xB1>(v);
    if constexpr (L >= 4) v += dpp<0x4E>(v);
    if constexpr (L >= 8) v += dpp<0x141>(v);
    if constexpr (L >= 16) v += dpp<0x140>(v);
    if constexpr (L >= 32) {
        const int i = __builtin_bit_cast(int, v);
        const auto r = __builtin_amdgcn_permlane16_swap(i, i, false, false);
        const uint32_t a = r[0], b = r[1];
        v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    }
    if constexpr (L >= 64) {
        const int i = __builtin_bit_cast(int, v);
        const auto r = __builtin_amdgcn_permlane32_swap(i, i, false, false);
        const uint32_t a = r[0], b = r[1];
        v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    }
    return v;
}

// Sums of N values over the L lanes of a row.  Above a wavefront the row is the
// workgroup's and the wavefronts meet in LDS: `region` alternates, so that one
// barrier per sum is enough (a region is written again only behind the next
// sum's barrier).
template <int L, int N>
__device__ inline void row_sum(float (&v)[N], float* lds, int& region) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_sum<(L < 64 ? L : 64)>(v[i]);
    if constexpr (L > 64) {
        constexpr int W = L / 64;
        float* at = lds + region * W * 2;
        region ^= 1;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) at[wave * 2 + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += at[w * 2 + i];
            v[i] = s;
        }
    }
}

// sigmoid(a) and 1 - sigmoid(a), both without cancellation.
__device__ inline void sigmoid2(float a, float& s, float& o) {
    const float t = __expf(-__builtin_fabsf(a));
    const float d = __builtin_amdgcn_rcpf(1.0f + t);
    const float small = t * d;
    s = a >= 0.0f ? d : small;
    o = a >= 0.0f ? small : d;
    if (a != a) s = o = a;
}

template <typename T>
struct JoinParams {
    const T *x, *z, *gate;
    const float *scale, *w_post, *w_pre;
    int64_t ldx, ldz, ldg, n_rows;
    int c, gate_kind;   // 0: none, 1: one per row, 2: one per channel
    float eps, inv_c;
    bool vec;
    bool stream;   // the backward's outputs go past the caches
    T *y, *h;
    const T *gy, *gh;
    T *gx, *gz, *ggate;
    float *gscale, *gpost, *gpre, *partial;
};

// The calls that training makes (all inputs and outputs there, everything on 16
// bytes) have code of their own without tests: a gate per channel, a gate per
// row.  kAny takes the rest by the parameters.  With the tests in the element
// loops, and lane sums through LDS, the gradients of 32768 x 2048 in bf16 took 291
// us and not 247, those of 16384 x 520 in fp32 92 and not 51.
enum Mode { kAny, kFull, kRow };
template <Mode M, typename T>
__device__ inline bool has_z(const JoinParams<T>& p) {
    return M != kAny || p.z;
}
template <Mode M, typename T>
__device__ inline bool has_pre(const JoinParams<T>& p) {
    return M != kAny || p.w_pre;
}
template <Mode M, typename T>
__device__ inline int gate_of(const JoinParams<T>& p) {
    return M == kFull ? 2 : (M == kRow ? 1 : p.gate_kind);
}
template <Mode M, typename T>
__device__ inline bool vec_of(const JoinParams<T>& p) {
    return M != kAny || p.vec;
}

constexpr int threads_of(int L) { return L > 256 ? L : 256; }

template <typename T, int L, int NV, Mode M>
__global__ __launch_bounds__(threads_of(L)) void zs_join_kernel(const JoinParams<T> p) {
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
        float y[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            Chunk<T>::unpack(load_chunk(p.x + row * p.ldx, l + j * L, c, vec_of<M>(p)), y[j]);
        if (has_z<M>(p)) {
            u32x4 zr[NV], ar[NV];
            float row_gate = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) zr[j] = load_chunk(p.z + row * p.ldz, l + j * L, c, vec_of<M>(p));
            if (gate_of<M>(p) == 2) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    ar[j] = load_chunk(p.gate + row * p.ldg, l + j * L, c, vec_of<M>(p));
            } else if (gate_of<M>(p) == 1 && live) {
                row_gate = float(p.gate[row * p.ldg]);
            }
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float z[V];
                Chunk<T>::unpack(zr[j], z);
#pragma unroll
                for (int i = 0; i < V; ++i) s[0] = __builtin_fmaf(z[i], z[i], s[0]);
            }
            row_sum<L>(s, lds, region);
            const float rz = 1.0f / sqrtf(__builtin_fmaf(s[0], p.inv_c, p.eps));
            float gate_s = 1.0f, gate_o = 0.0f;
            if (gate_of<M>(p) == 1) sigmoid2(row_gate, gate_s, gate_o);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float z[V], a[V], sc[V], wp[V];
                Chunk<T>::unpack(zr[j], z);
                load_param<V>(p.scale, l + j * L, c, vec_of<M>(p), sc);
                load_param<V>(p.w_post, l + j * L, c, vec_of<M>(p), wp);
                if (gate_of<M>(p) == 2) Chunk<T>::unpack(ar[j], a);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float g = gate_s, o;
                    if (gate_of<M>(p) == 2) sigmoid2(a[i], g, o);
                    y[j][i] = __builtin_fmaf(sc[i] * g, z[i] * rz * wp[i], y[j][i]);
                }
                if (live) store_chunk(p.y + row * p.c, l + j * L, c, vec_of<M>(p), Chunk<T>::pack(y[j]));
            }
        }
        if (has_pre<M>(p)) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) s[0] = __builtin_fmaf(y[j][i], y[j][i], s[0]);
            row_sum<L>(s, lds, region);
            const float ry = 1.0f / sqrtf(__builtin_fmaf(s[0], p.inv_c, p.eps));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float w[V];
                load_param<V>(p.w_pre, l + j * L, c, vec_of<M>(p), w);
#pragma unroll
                for (int i = 0; i < V; ++i) w[i] = y[j][i] * ry * w[i];
                if (live) store_chunk(p.h + row * p.c, l + j * L, c, vec_of<M>(p), Chunk<T>::pack(w));
            }
        }
    }
}

// Workgroups of the backward on a compute unit: as many as the registers of a
// lane's part of a row (and, with a gate per channel, its sigmoids) leave room
// for without spilling.
template <typename T, int L, int NV, Mode M>
constexpr int resident() {
    constexpr int held = NV * Chunk<T>::V;
    if (L > 256) return 1;
    return held <= 4 ? 4 : (held <= 8 || (held <= 12 && M == kRow) ? 3 : 2);
}

// A lane's part of a row's inputs as they lie in memory.
template <int NV>
struct RowInputs {
    u32x4 z[NV], x[NV], gate[NV], gy[NV], gh[NV];
    float row_gate;
};
template <typename T, int L, int NV, Mode M>
__device__ inline RowInputs<NV> load_row(const JoinParams<T>& p, int64_t row, int l) {
    RowInputs<NV> r;
    const bool live = row < p.n_rows, vec = vec_of<M>(p);
    const int c = live ? p.c : 0;
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int at = l + j * L;
        r.z[j] = r.x[j] = r.gate[j] = r.gy[j] = r.gh[j] = zero;
        if (at * Chunk<T>::V < c) {
            r.x[j] = load_chunk<T, true>(p.x + row * p.ldx, at, c, vec);
            if (has_z<M>(p)) r.z[j] = load_chunk<T, true>(p.z + row * p.ldz, at, c, vec);
            if (gate_of<M>(p) == 2) r.gate[j] = load_chunk<T, true>(p.gate + row * p.ldg, at, c, vec);
            if (M != kAny || p.gy) r.gy[j] = load_chunk<T, true>(p.gy + row * p.c, at, c, vec);
            if (M != kAny || p.gh) r.gh[j] = load_chunk<T, true>(p.gh + row * p.c, at, c, vec);
        }
    }
    r.row_gate = gate_of<M>(p) == 1 && live ? float(p.gate[row * p.ldg]) : 0.0f;
    return r;
}

template <typename T, int L, int NV, Mode M>
__global__ __launch_bounds__(threads_of(L), (resident<T, L, NV, M>())) void zs_join_bwd_kernel(
    const JoinParams<T> p) {
    constexpr int V = Chunk<T>::V;
    constexpr int kThreads = threads_of(L), kRowsOf = kThreads / L;
    __shared__ float lds[2 * (L > 64 ? L / 64 : 1) * 2];
    __shared__ float sums[kRowsOf > 1 ? kThreads * V : 1];
    int region = 0;
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    float acc[3][NV][V];   // scale, w_post, w_pre
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[q][j][i] = 0.0f;
    // a lane with one chunk of a row has registers left to load the next row's
    // while this one's is used
    constexpr bool kAhead = NV == 1;
    RowInputs<NV> next;
    if constexpr (kAhead) next = load_row<T, L, NV, M>(p, int64_t(blockIdx.x) * kRowsOf + slot, l);
    for (int64_t base = int64_t(blockIdx.x) * kRowsOf; base < p.n_rows;
         base += int64_t(gridDim.x) * kRowsOf) {
        const int64_t row = base + slot;
        const bool live = row < p.n_rows;
        const int c = live ? p.c : 0;
        const RowInputs<NV> in = kAhead ? next : load_row<T, L, NV, M>(p, row, l);
        if constexpr (kAhead) next = load_row<T, L, NV, M>(p, row + int64_t(gridDim.x) * kRowsOf, l);
        float y[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) Chunk<T>::unpack(in.x[j], y[j]);
        float rz = 0.0f, gate_s = 1.0f, gate_o = 0.0f;
        if (has_z<M>(p)) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float z[V];
                Chunk<T>::unpack(in.z[j], z);
#pragma unroll
                for (int i = 0; i < V; ++i) s[0] = __builtin_fmaf(z[i], z[i], s[0]);
            }
            row_sum<L>(s, lds, region);
            rz = 1.0f / sqrtf(__builtin_fmaf(s[0], p.inv_c, p.eps));
            if (gate_of<M>(p) == 1) sigmoid2(in.row_gate, gate_s, gate_o);
        }
        float s2[2] = {0.0f, 0.0f};   // y^2, t y
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = l + j * L;
            if (has_z<M>(p)) {
                float z[V], a[V], sc[V], wp[V];
                Chunk<T>::unpack(in.z[j], z);
                load_param<V>(p.scale, at, c, vec_of<M>(p), sc);
                load_param<V>(p.w_post, at, c, vec_of<M>(p), wp);
                if (gate_of<M>(p) == 2) Chunk<T>::unpack(in.gate[j], a);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float g = gate_s, o;
                    if (gate_of<M>(p) == 2) sigmoid2(a[i], g, o);
                    y[j][i] = __builtin_fmaf(sc[i] * g, z[i] * rz * wp[i], y[j][i]);
                }
            }
            if (has_pre<M>(p)) {
                float gh[V], w[V];
                Chunk<T>::unpack(in.gh[j], gh);
                load_param<V>(p.w_pre, at, c, vec_of<M>(p), w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s2[0] = __builtin_fmaf(y[j][i], y[j][i], s2[0]);
                    s2[1] = __builtin_fmaf(gh[i] * w[i], y[j][i], s2[1]);
                }
            }
        }
        float ry = 0.0f, my = 0.0f;   // my = mean(t yn)
        if (has_pre<M>(p)) {
            row_sum<L>(s2, lds, region);
            ry = 1.0f / sqrtf(__builtin_fmaf(s2[0], p.inv_c, p.eps));
            my = ry * (s2[1] * p.inv_c);
        }
        float s3[2] = {0.0f, 0.0f};   // r zn, q u (1 - s)
        float gx[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = l + j * L;
            Chunk<T>::unpack(in.gy[j], gx[j]);
            if (has_pre<M>(p)) {
                float gh[V], w[V];
                Chunk<T>::unpack(in.gh[j], gh);
                load_param<V>(p.w_pre, at, c, vec_of<M>(p), w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float yn = y[j][i] * ry;
                    acc[2][j][i] = __builtin_fmaf(gh[i], yn, acc[2][j][i]);
                    gx[j][i] = __builtin_fmaf(ry, gh[i] * w[i], gx[j][i]) - (my * ry) * yn;
                }
            }
            if (live) store_chunk(p.gx + row * p.c, at, c, vec_of<M>(p), Chunk<T>::pack(gx[j]), p.stream);
            if (has_z<M>(p)) {
                float z[V], a[V], sc[V], wp[V], ga[V];
                Chunk<T>::unpack(in.z[j], z);
                load_param<V>(p.scale, at, c, vec_of<M>(p), sc);
                load_param<V>(p.w_post, at, c, vec_of<M>(p), wp);
                if (gate_of<M>(p) == 2) Chunk<T>::unpack(in.gate[j], a);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float g = gate_s, o = gate_o;
                    if (gate_of<M>(p) == 2) sigmoid2(a[i], g, o);
                    const float zn = z[i] * rz, u = zn * wp[i];
                    const float b = gx[j][i] * g, q = b * sc[i], r = q * wp[i];
                    acc[0][j][i] = __builtin_fmaf(b, u, acc[0][j][i]);
                    acc[1][j][i] = __builtin_fmaf(q, zn, acc[1][j][i]);
                    s3[0] = __builtin_fmaf(r, zn, s3[0]);
                    ga[i] = q * u * o;
                    s3[1] += ga[i];
                    gx[j][i] = r;
                }
                if (gate_of<M>(p) == 2 && live)
                    store_chunk(p.ggate + row * p.c, at, c, vec_of<M>(p), Chunk<T>::pack(ga), p.stream);
            }
        }
        if (has_z<M>(p)) {
            row_sum<L>(s3, lds, region);
            if (gate_of<M>(p) == 1 && live && l == 0) p.ggate[row] = T(s3[1]);
            const float mz = s3[0] * p.inv_c;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float z[V];
                Chunk<T>::unpack(in.z[j], z);
#pragma unroll
                for (int i = 0; i < V; ++i) z[i] = rz * (gx[j][i] - z[i] * rz * mz);
                if (live) store_chunk(p.gz + row * p.c, l + j * L, c, vec_of<M>(p), Chunk<T>::pack(z), p.stream);
            }
        }
    }
    // sums over the workgroup's row slots, then out: [3][c] per workgroup.  A single
    // workgroup's are the gradients (not where a workgroup takes a row at a time: that
    // would be one row, and the choice costs those kernels spilled registers).
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        float* out = p.partial + (int64_t(blockIdx.x) * 3 + q) * p.c;
        if (kRowsOf > 1 && gridDim.x == 1) out = q == 0 ? p.gscale : (q == 1 ? p.gpost : p.gpre);
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
                    if (ch < p.c && out) out[ch] = s;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int ch = (j * L + l) * V + i;
                    if (ch < p.c && out) out[ch] = acc[q][j][i];
                }
            }
        }
    }
}

// Adds the workgroups' partial sums in order: 32 columns a workgroup, 32 lanes
// of partial rows each, joined in LDS.
__global__ __launch_bounds__(1024) void zs_join_sum_kernel(const float* partial, int count, int c,
                                                           float* gscale, float* gpost,
                                                           float* gpre) {
    __shared__ float lds[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    float s = 0.0f;
    if (col < 3 * c) {
#pragma unroll 4
        for (int i = part; i < count; i += 32) s += partial[int64_t(i) * 3 * c + col];
    }
    lds[part][threadIdx.x & 31] = s;
    __syncthreads();
    if (part == 0 && col < 3 * c) {
        s = 0.0f;
        for (int i = 0; i < 32; ++i) s += lds[i][threadIdx.x];
        float* out = col < c ? gscale : (col < 2 * c ? gpost : gpre);
        if (out) out[col % c] = s;
    }
}

template <typename T>
JoinParams<T> params(const JoinArgs& a) {
    constexpr int V = Chunk<T>::V;
    JoinParams<T> p{};
    p.x = static_cast<const T*>(a.x), p.z = static_cast<const T*>(a.z);
    p.gate = static_cast<const T*>(a.gate);
    p.scale = a.scale, p.w_post = a.w_post, p.w_pre = a.w_pre;
    p.ldx = a.ldx, p.ldz = a.ldz, p.ldg = a.ldg, p.n_rows = a.n_rows;
    p.c = a.c;
    // a gate per channel of one channel is the gate per row
    p.gate_kind = a.gate_width == 0 ? 0 : (a.gate_width == 1 ? 1 : 2);
    p.eps = a.eps, p.inv_c = 1.0f / float(a.c);
    p.y = static_cast<T*>(a.y), p.h = static_cast<T*>(a.h);
    p.gy = static_cast<const T*>(a.gy), p.gh = static_cast<const T*>(a.gh);
    p.gx = static_cast<T*>(a.gx), p.gz = static_cast<T*>(a.gz), p.ggate = static_cast<T*>(a.ggate);
    p.gscale = a.gscale, p.gpost = a.gpost, p.gpre = a.gpre, p.partial = a.partial;
    const auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    p.vec = a.c % V == 0 && a.ldx % V == 0 && on16(a.x) && on16(a.y) && on16(a.h) && on16(a.gy) &&
            on16(a.gh) && on16(a.gx) && on16(a.gz) && on16(a.scale) && on16(a.w_post) &&
            on16(a.w_pre);
    // Gradients that fill half of the memory-side cache by themselves are written past
    // the caches (32768 x 2048 in bf16, 134 MB each: 240 us, 246 otherwise); smaller
    // ones are there for whoever reads them next (16384 x 520 in fp32, 34 MB: 49 past
    // the caches, 48 otherwise).  The backward's inputs, read once, are always read
    // past them (247 and 51 us otherwise).
    p.stream = a.n_rows * a.c * int64_t(sizeof(T)) >= (int64_t(128) << 20);
    if (a.z) p.vec = p.vec && a.ldz % V == 0 && on16(a.z);
    if (p.gate_kind == 2)
        p.vec = p.vec && a.ldg % V == 0 && on16(a.gate) && on16(a.ggate);
    return p;
}

constexpr int64_t kMaxPartials = 1024;

template <typename T, int L, int NV, Mode M>
hipError_t run_mode(const JoinParams<T>& p, bool backward, hipStream_t stream) {
    constexpr int rows = threads_of(L) / L;
    const int64_t want = (p.n_rows + rows - 1) / rows;
    if (!backward) {
        const unsigned grid = unsigned(want < 8192 ? want : 8192);
        zs_join_kernel<T, L, NV, M><<<grid, threads_of(L), 0, stream>>>(p);
        return hipGetLastError();
    }
    // one round of workgroups that all run at once
    constexpr int64_t cap = 256 * resident<T, L, NV, M>();
    static_assert(cap <= kMaxPartials, "partial sums for every workgroup");
    const unsigned grid = unsigned(want < cap ? want : cap);
    if (grid > 0) {
        zs_join_bwd_kernel<T, L, NV, M><<<grid, threads_of(L), 0, stream>>>(p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess || (rows > 1 && grid == 1)) return err;
    }
    zs_join_sum_kernel<<<(3 * p.c + 31) / 32, 1024, 0, stream>>>(p.partial, int(grid), p.c,
                                                                 p.gscale, p.gpost, p.gpre);
    return hipGetLastError();
}

template <typename T, int L, int NV>
hipError_t run(const JoinArgs& a, bool backward, hipStream_t stream) {
    const JoinParams<T> p = params<T>(a);
    const bool all = p.vec && p.z && p.w_pre && (!backward || (p.gy && p.gh));
    // (the widest fp32 rows leave no registers for the sigmoids of a gate per channel)
    if constexpr (sizeof(T) == 2 || L <= 256)
        if (all && p.gate_kind == 2) return run_mode<T, L, NV, kFull>(p, backward, stream);
    if (all && p.gate_kind == 1) return run_mode<T, L, NV, kRow>(p, backward, stream);
    return run_mode<T, L, NV, kAny>(p, backward, stream);
}

// Lanes and chunks per lane by the row's width in chunks: the fewest lanes that
// hold a row in one chunk each up to a wavefront, then two or three chunks a
// lane, then a workgroup (bf16 chunks are eight values: three of them a lane
// spill in the backward).
template <typename T>
hipError_t dispatch(const JoinArgs& a, bool backward, hipStream_t stream) {
    const int chunks = (a.c + Chunk<T>::V - 1) / Chunk<T>::V;
    if (chunks <= 1) return run<T, 1, 1>(a, backward, stream);
    if (chunks <= 2) return run<T, 2, 1>(a, backward, stream);
    if (chunks <= 4) return run<T, 4, 1>(a, backward, stream);
    if (chunks <= 8) return run<T, 8, 1>(a, backward, stream);
    if (chunks <= 16) return run<T, 16, 1>(a, backward, stream);
    if (chunks <= 32) return run<T, 32, 1>(a, backward, stream);
    if (chunks <= 64) return run<T, 64, 1>(a, backward, stream);
    if (chunks <= 128) return run<T, 64, 2>(a, backward, stream);
    if constexpr (sizeof(T) == 4) {
        if (chunks <= 192) return run<T, 64, 3>(a, backward, stream);
        if (chunks <= 256) return run<T, 256, 1>(a, backward, stream);
        if (chunks <= 512) return run<T, 256, 2>(a, backward, stream);
        if (chunks <= 1024) return run<T, 256, 4>(a, backward, stream);
        return run<T, 512, 4>(a, backward, stream);
    } else {
        if (chunks <= 256) return run<T, 256, 1>(a, backward, stream);
        if (chunks <= 512) return run<T, 256, 2>(a, backward, stream);
        return run<T, 512, 2>(a, backward, stream);
    }
}

}  // namespace

size_t join_workspace(int64_t n_rows, int64_t c) {
    int64_t parts = n_rows < kMaxPartials ? n_rows : kMaxPartials;
    return size_t(parts * 3 * c * 4);
}

hipError_t launch_join(const JoinArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, false, stream) : dispatch<float>(a, false, stream);
}

hipError_t launch_join_backward(const JoinArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, true, stream) : dispatch<float>(a, true, stream);
}

}  // namespace zs
