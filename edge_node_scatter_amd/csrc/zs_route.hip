// Routing of rows to experts and its gradient, gfx950.
//
//   s = softmax(x) or sigmoid(x) of a row, q = s + bias;  of the experts that are there
//   (x and bias above -inf) in the top_groups groups of largest score (the sum of
//   the group's best one or two q) the k of largest q, ties to the lowest index;
//   w_j = a s_ij, or a p_j with p_j = s_ij / sum_l s_il
//
// backward, the choice held fixed, over the slots that hold an expert:
//   renormalised: dx_ij = a p_j (gw_j - sum_l gw_l p_l), times 1 - s_ij for sigmoid
//   sigmoid:      dx_ij = a gw_j s_ij (1 - s_ij)
//   softmax:      dx_e = [e chosen] a gw_j s_e - s_e sum_l a gw_l s_il
//
// A row lies in the registers of L lanes, NV consecutive experts each, so that of
// equal values the lowest lane's first one has the lowest index.
#include "zs_layers_internal.h"
#include "zs_row.h"

namespace zs {

namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

template <typename T>
struct RouteParams {
    const T* x;
    const float* bias;
    int64_t ldx, n_rows;
    int n, k, groups, top_groups, best;
    bool sigmoid, renormalise;
    float scale;
    float* weight;
    int64_t* expert;
    const float* gw;
    const int64_t* chosen;
    T* gx;
};

// Over the L lanes of a row, in all of them.
template <int L>
__device__ inline float row_max(float v) {
#pragma unroll
    for (int d = 1; d < L; d *= 2) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}
template <int L>
__device__ inline double row_max(double v) {
#pragma unroll
    for (int d = 1; d < L; d *= 2) v = fmax(v, __shfl_xor(v, d, 64));
    return v;
}
template <int L>
__device__ inline double row_add(double v) {
#pragma unroll
    for (int d = 1; d < L; d *= 2) v += __shfl_xor(v, d, 64);
    return v;
}
// The bits of the row's lanes, the first lane's lowest.
template <int L>
__device__ inline uint64_t row_ballot(bool b) {
    const uint64_t all = __ballot(b);
    if constexpr (L == 64) return all;
    return all >> ((threadIdx.x & 63) / L * L) & ((uint64_t(1) << (L & 63)) - 1);
}

// Bytes of LDS of a row: shares (8), logits (4) and indices (4) of the slots, and with
// groups the experts' q (8), the groups' scores (8) and whether they stay (4).
__host__ __device__ inline int row_bytes(int n, int k, int groups) {
    return k * 16 + (groups > 1 ? n * 8 + (groups * 12 + 7) / 8 * 8 : 0);
}

template <typename T, int L, int NV>
__global__ __launch_bounds__(kThreads) void zs_route_kernel(const RouteParams<T> p) {
    extern __shared__ char lds[];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    char* mine = lds + slot * row_bytes(p.n, p.k, p.groups);
    double* share = reinterpret_cast<double*>(mine);
    double* q_of = share + p.k;
    double* score = q_of + (p.groups > 1 ? p.n : 0);
    float* xs = reinterpret_cast<float*>(score + (p.groups > 1 ? p.groups : 0));
    int* id = reinterpret_cast<int*>(xs + p.k);
    int* stays = id + p.k;
    for (int64_t base = int64_t(blockIdx.x) * (kThreads / L); base < p.n_rows;
         base += int64_t(gridDim.x) * (kThreads / L)) {
        const int64_t row = base + slot;
        const bool live = row < p.n_rows;
        float x[NV];
        double key[NV];
        bool there[NV];
        bool bad = false;
        float top = -kInf;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = l * NV + i;
            x[i] = live && e < p.n ? float(p.x[row * p.ldx + e]) : -kInf;
            bad |= x[i] != x[i];
            top = fmaxf(top, x[i]);
            there[i] = x[i] > -kInf;
            key[i] = x[i];
        }
        if (!p.sigmoid) {
            top = row_max<L>(top);
            bad |= top == kInf;
        }
        bad = row_ballot<L>(bad) != 0;
        double total = 1.0;
        if (!p.sigmoid && (p.bias || p.groups > 1 || !p.renormalise)) {
            total = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) total += there[i] ? exp(double(x[i]) - double(top)) : 0.0;
            total = row_add<L>(total);
        }
        if (p.bias || p.groups > 1) {
            double q[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = l * NV + i;
                q[i] = p.sigmoid ? 1.0 / (1.0 + exp(-double(x[i])))
                                 : exp(double(x[i]) - double(top)) / total;
                if (p.bias && e < p.n) {
                    const float b = p.bias[e];
                    there[i] = there[i] && b > -kInf;
                    q[i] += double(b);
                }
                if (!there[i]) q[i] = -double(kInf);
            }
            if (p.groups > 1) {
                const int per = p.n / p.groups;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (l * NV + i < p.n) q_of[l * NV + i] = q[i];
                wave_lds_sync();
                for (int g = l; g < p.groups; g += L) {
                    double a = -double(kInf), b = -double(kInf);
                    for (int e = g * per; e < (g + 1) * per; ++e) {
                        const double v = q_of[e];
                        b = fmax(b, fmin(a, v));
                        a = fmax(a, v);
                    }
                    score[g] = p.best == 2 && b > -double(kInf) ? a + b : a;
                }
                wave_lds_sync();
                for (int g = l; g < p.groups; g += L) {
                    int before = 0;
                    const double s = score[g];
                    for (int h = 0; h < p.groups; ++h)
                        before += score[h] > s || (score[h] == s && h < g);
                    stays[g] = before < p.top_groups;
                }
                wave_lds_sync();
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int e = l * NV + i;
                    there[i] = there[i] && stays[(e < p.n ? e : 0) / per];
                }
            }
            if (p.bias)
#pragma unroll
                for (int i = 0; i < NV; ++i) key[i] = q[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (!there[i] || bad) key[i] = -double(kInf);
        // k rounds: the row's largest key, from the lowest lane and place that holds it
        for (int r = 0; r < p.k; ++r) {
            double best = key[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < NV; ++i)
                if (key[i] > best) best = key[i], at = i;
            const double m = row_max<L>(best);
            const uint64_t who = row_ballot<L>(best == m && m > -double(kInf));
            if (who == 0) {
                if (l == 0) id[r] = p.n, xs[r] = -kInf;
            } else if (l == __ffsll(static_cast<unsigned long long>(who)) - 1) {
                id[r] = l * NV + at;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (i == at) xs[r] = x[i], key[i] = -double(kInf);
            }
        }
        wave_lds_sync();
        // weights from the chosen logits
        float high = -kInf;
        if (p.renormalise && !p.sigmoid)
            for (int r = 0; r < p.k; ++r) high = fmaxf(high, xs[r]);
        for (int r = l; r < p.k; r += L) {
            const double v = xs[r];
            double s = 0.0;
            if (id[r] < p.n) {
                if (p.sigmoid) s = 1.0 / (1.0 + exp(-v));
                else if (p.renormalise) s = exp(v - double(high));
                else s = exp(v - double(top)) / total;
            }
            share[r] = s;
        }
        wave_lds_sync();
        double sum = 1.0;
        if (p.renormalise) {
            sum = 0.0;
            for (int r = 0; r < p.k; ++r) sum += share[r];
        }
        for (int r = l; r < p.k; r += L) {
            if (!live) continue;
            const float w = float(double(p.scale) * (sum > 0.0 ? share[r] / sum : 0.0));
            p.weight[row * p.k + r] = bad ? __builtin_nanf("") : w;
            p.expert[row * p.k + r] = id[r];
        }
        wave_lds_sync();   // before the next row's choice is written
    }
}

// Bytes of LDS of a row in the backward: a slot's share and gradient (8 each), its
// index (4).
__host__ __device__ inline int back_bytes(int k) { return k * 24; }

template <typename T, int L, int NV>
__global__ __launch_bounds__(kThreads) void zs_route_bwd_kernel(const RouteParams<T> p) {
    extern __shared__ char lds[];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    double* share = reinterpret_cast<double*>(lds + slot * back_bytes(p.k));
    double* grad = share + p.k;
    int* id = reinterpret_cast<int*>(grad + p.k);
    const bool full = !p.sigmoid && !p.renormalise;   // every logit has a part in the weights
    for (int64_t base = int64_t(blockIdx.x) * (kThreads / L); base < p.n_rows;
         base += int64_t(gridDim.x) * (kThreads / L)) {
        const int64_t row = base + slot;
        const bool live = row < p.n_rows;
        const T* x = p.x + row * p.ldx;
        float s[NV];
        float top = -kInf;
        double total = 1.0;
        if (full) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = l * NV + i;
                s[i] = live && e < p.n ? float(x[e]) : -kInf;
                top = fmaxf(top, s[i]);
            }
            top = row_max<L>(top);
            total = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const double v = l * NV + i < p.n ? exp(double(s[i]) - double(top)) : 0.0;
                total += v;
                s[i] = float(v);
            }
            total = row_add<L>(total);
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] = float(double(s[i]) / total);
        }
        // the slots' logits, the largest of them, and their shares
        float high = -kInf;
        for (int r = l; r < p.k; r += L) {
            const int64_t e = live ? p.chosen[row * p.k + r] : -1;
            const bool in = e >= 0 && e < p.n;
            id[r] = in ? int(e) : -1;
            const float v = in ? float(x[e]) : -kInf;
            share[r] = v;
            high = fmaxf(high, v);
            grad[r] = in ? double(p.gw[row * p.k + r]) * double(p.scale) : 0.0;
        }
        if (p.renormalise && !p.sigmoid) high = row_max<L>(high);
        wave_lds_sync();
        for (int r = l; r < p.k; r += L) {
            const double v = share[r];
            double w = 0.0;
            if (id[r] >= 0) {
                if (p.sigmoid) w = 1.0 / (1.0 + exp(-v));
                else if (p.renormalise) w = exp(v - double(high));
                else w = exp(v - double(top)) / total;
            }
            share[r] = w;
        }
        wave_lds_sync();
        double sum = 1.0;
        bool any = false;
        if (p.renormalise) sum = 0.0;
        for (int r = 0; r < p.k; ++r) {
            if (p.renormalise) sum += share[r];
            any |= id[r] >= 0;
        }
        if (!(sum > 0.0)) sum = 1.0;   // all shares are 0
        double mean = 0.0;   // of the gradients with the shares
        if (p.renormalise || full)
            for (int r = 0; r < p.k; ++r) mean += grad[r] * (share[r] / sum);
        wave_lds_sync();
        for (int r = l; r < p.k; r += L) {
            const double w = share[r], g = grad[r];
            const double d = p.renormalise ? w / sum * (g - mean) : g * w;
            grad[r] = p.sigmoid ? d * (1.0 - w) : d;
        }
        wave_lds_sync();
        float out[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) out[i] = full && any ? -s[i] * float(mean) : 0.0f;
        for (int r = 0; r < p.k; ++r) {
            const float d = float(grad[r]);
            const int at = id[r] - l * NV;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i == at) out[i] += d;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = l * NV + i;
            if (live && e < p.n) p.gx[row * p.n + e] = T(out[i]);
        }
        wave_lds_sync();   // before the next row's slots are written
    }
}

template <typename T, int L, int NV>
hipError_t run(const RouteArgs& a, bool backward, hipStream_t stream) {
    RouteParams<T> p{};
    p.x = static_cast<const T*>(a.x), p.bias = a.bias, p.ldx = a.ldx, p.n_rows = a.n_rows;
    p.n = a.n, p.k = a.r.k, p.groups = a.r.groups, p.top_groups = a.r.top_groups;
    p.best = a.r.best, p.sigmoid = a.r.sigmoid != 0, p.renormalise = a.r.renormalise != 0;
    p.scale = a.r.scale, p.weight = a.weight, p.expert = a.expert;
    p.gw = a.gw, p.chosen = a.chosen, p.gx = static_cast<T*>(a.gx);
    constexpr int rows = kThreads / L;
    const int64_t want = (a.n_rows + rows - 1) / rows;
    const unsigned grid = unsigned(want < 1 << 20 ? want : 1 << 20);
    if (backward)
        zs_route_bwd_kernel<T, L, NV>
            <<<grid, kThreads, size_t(rows) * back_bytes(p.k), stream>>>(p);
    else
        zs_route_kernel<T, L, NV>
            <<<grid, kThreads, size_t(rows) * row_bytes(p.n, p.k, p.groups), stream>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t dispatch(const RouteArgs& a, bool backward, hipStream_t stream) {
    if (a.n <= 8) return run<T, 8, 1>(a, backward, stream);
    if (a.n <= 32) return run<T, 8, 4>(a, backward, stream);
    if (a.n <= 64) return run<T, 16, 4>(a, backward, stream);
    if (a.n <= 128) return run<T, 32, 4>(a, backward, stream);
    if (a.n <= 256) return run<T, 64, 4>(a, backward, stream);
    if (a.n <= 512) return run<T, 64, 8>(a, backward, stream);
    return run<T, 64, 16>(a, backward, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, false, stream) : dispatch<float>(a, false, stream);
}

hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? dispatch<__bf16>(a, true, stream) : dispatch<float>(a, true, stream);
}

}  // namespace zs
