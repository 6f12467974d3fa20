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
    int group_factor;   // e * group_factor >> 20 is the group of expert e
    bool sigmoid, renormalise;
    float scale;
    float* weight;
    int64_t* expert;
    const float* gw;
    const int64_t* chosen;
    T* gx;
};

// Value of the lane that a DPP control picks within 16 lanes.
template <int CTRL>
__device__ inline float from_lane(float v) {
    return dpp<CTRL>(v);
}
template <int CTRL>
__device__ inline double from_lane(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(b)), CTRL, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(b >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
// The two halves of 32 or 64 lanes, in every lane of them.
template <bool WIDE>
__device__ inline void halves(uint32_t v, uint32_t& a, uint32_t& b) {
    if constexpr (WIDE) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        a = r[0], b = r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        a = r[0], b = r[1];
    }
}
template <bool WIDE>
__device__ inline void halves(float v, float& a, float& b) {
    uint32_t x, y;
    halves<WIDE>(__builtin_bit_cast(uint32_t, v), x, y);
    a = __builtin_bit_cast(float, x), b = __builtin_bit_cast(float, y);
}
template <bool WIDE>
__device__ inline void halves(double v, double& a, double& b) {
    const uint64_t bits = __builtin_bit_cast(uint64_t, v);
    uint32_t al, bl, ah, bh;
    halves<WIDE>(uint32_t(bits), al, bl);
    halves<WIDE>(uint32_t(bits >> 32), ah, bh);
    a = __builtin_bit_cast(double, uint64_t(ah) << 32 | al);
    b = __builtin_bit_cast(double, uint64_t(bh) << 32 | bl);
}
// f over the L lanes of a row, in all of them, without LDS.
template <int L, typename V, typename F>
__device__ inline V over_row(V v, F f) {
    v = f(v, from_lane<0xB1>(v));
    v = f(v, from_lane<0x4E>(v));
    v = f(v, from_lane<0x141>(v));
    if constexpr (L >= 16) v = f(v, from_lane<0x140>(v));
    if constexpr (L >= 32) {
        V a, b;
        halves<false>(v, a, b);
        v = f(a, b);
    }
    if constexpr (L >= 64) {
        V a, b;
        halves<true>(v, a, b);
        v = f(a, b);
    }
    return v;
}
template <int L, typename V>
__device__ inline V row_max(V v) {
    return over_row<L>(v, [](V a, V b) { return a > b ? a : b; });
}
template <int L>
__device__ inline float row_max(float v) {
    return over_row<L>(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
template <int L>
__device__ inline double row_add(double v) {
    return over_row<L>(v, [](double a, double b) { return a + b; });
}
// The bits of the row's lanes, the first lane's lowest.
template <int L>
__device__ inline uint64_t row_ballot(bool b) {
    const uint64_t all = __ballot(b);
    if constexpr (L == 64) return all;
    return all >> ((threadIdx.x & 63) / L * L) & ((uint64_t(1) << (L & 63)) - 1);
}

// NV logits from an address of any alignment; zeros behind the row's end.
template <typename T, int NV>
__device__ inline void load_logits(const T* row, int at, int n, float (&x)[NV]) {
    if (at + NV <= n) {
        T raw[NV];
        __builtin_memcpy(raw, row + at, sizeof raw);
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = float(raw[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = at + i < n ? float(row[at + i]) : 0.0f;
    }
}

// The largest and second largest of two such pairs.
struct Best2 {
    float a, b;
};
__device__ inline Best2 join(Best2 p, float a, float b) {
    return Best2{__builtin_fmaxf(p.a, a),
                 __builtin_fmaxf(__builtin_fminf(p.a, a), __builtin_fmaxf(p.b, b))};
}

// Bytes of LDS of a row: shares (8), logits (4) and indices (4) of the slots, and with
// groups the experts' q (8), the groups' scores (8) and whether they stay (4).
__host__ __device__ inline int row_bytes(int n, int k, int groups) {
    return k * 16 + (groups > 1 ? n * 8 + (groups * 12 + 7) / 8 * 8 : 0);
}

// The k experts of largest key, by rounds: the row's largest key, from the lowest lane
// and place that holds it.  The chosen indices and logits go to LDS, n where no key
// is left.  Returns whether two keys that follow each other, up to the first that is not
// chosen, are no further apart than tol (tol < 0: not asked).
template <int L, int NV, typename K>
__device__ inline bool choose(K (&key)[NV], const float (&x)[NV], int l, int n, int k, K tol,
                              int* id, float* xs) {
    constexpr K none = -K(kInf);
    K best = none, before = K(kInf);
    int at = 0;
    const auto find = [&] {
        best = key[0], at = 0;
#pragma unroll
        for (int i = 1; i < NV; ++i)
            if (key[i] > best) best = key[i], at = i;
    };
    find();
    bool close = false;
    for (int r = 0; r < k; ++r) {
        const K m = row_max<L>(best);
        if (tol >= K(0)) close |= before - m <= tol;
        before = m;
        const uint64_t who = row_ballot<L>(best == m && m > none);
        const int lane = who ? __builtin_ctzll(who) : -1;
        if (l == lane) {
            id[r] = l * NV + at;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i == at) xs[r] = x[i], key[i] = none;
            find();
        }
        if (lane < 0 && l == 0) id[r] = n, xs[r] = -kInf;
    }
    if (tol >= K(0)) close |= before - row_max<L>(best) <= tol;
    return close;
}

template <typename T, int L, int NV>
__global__ __launch_bounds__(kThreads) void zs_route_kernel(const RouteParams<T> p) {
    extern __shared__ char lds[];
    const int l = threadIdx.x % L, slot = threadIdx.x / L, e0 = l * NV;
    char* mine = lds + slot * row_bytes(p.n, p.k, p.groups);
    double* share = reinterpret_cast<double*>(mine);
    double* q_of = share + p.k;
    double* score = q_of + (p.groups > 1 ? p.n : 0);
    float* xs = reinterpret_cast<float*>(score + (p.groups > 1 ? p.groups : 0));
    int* id = reinterpret_cast<int*>(xs + p.k);
    int* stays = id + p.k;
    const int per = p.n / p.groups;
    const bool ranked = p.bias || p.groups > 1;   // by more than the logits
    for (int64_t base = int64_t(blockIdx.x) * (kThreads / L); base < p.n_rows;
         base += int64_t(gridDim.x) * (kThreads / L)) {
        const int64_t row = base + slot;
        const bool live = row < p.n_rows;
        float x[NV], b[NV];
        bool there[NV];
        bool bad = false;
        float top = -kInf;
        load_logits<T, NV>(p.x + row * p.ldx, e0, live ? p.n : 0, x);
        if (p.bias) load_logits<float, NV>(p.bias, e0, p.n, b);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            bad |= x[i] != x[i];
            there[i] = live && e0 + i < p.n && x[i] > -kInf;
            if (!there[i]) x[i] = -kInf;
            if (p.bias) there[i] = there[i] && b[i] > -kInf;
            else b[i] = 0.0f;
            top = __builtin_fmaxf(top, x[i]);
        }
        if (!p.sigmoid) {
            top = row_max<L>(top);
            bad |= top == kInf;
        }
        bad = row_ballot<L>(bad) != 0;
        // scores in fp32, and how far two sums of a score and a bias may lie apart that
        // fp64 might order otherwise
        float s[NV], most = 1.0f;
        double total = 1.0;
        if (!p.sigmoid && (ranked || !p.renormalise)) {
            total = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i] = x[i] > -kInf ? expf(x[i] - top) : 0.0f;
                total += double(s[i]);
            }
            total = row_add<L>(total);
            most = total > 0.0 ? 1.0f / float(total) : 1.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] *= most;
        } else if (ranked) {
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
        }
        bool close = false;
        float key[NV];
        float tol = -1.0f;
        if (ranked) {
            float size = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i] = there[i] ? s[i] + b[i] : -kInf;
                size = __builtin_fmaxf(size, there[i] ? __builtin_fabsf(s[i]) : 0.0f);
            }
            size = row_max<L>(size);
            tol = most * 0x1p-19f + size * 0x1p-22f;
            close = !(tol < kInf);
        }
        if (p.groups > 1) {
            // lanes that hold a group, if whole lanes do and DPP joins them
            const int lanes = per / NV;
            float mine_score;
            const bool whole = per % NV == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0;
            float* score32 = reinterpret_cast<float*>(score);
            if (whole) {
                Best2 t{s[0], -kInf};
#pragma unroll
                for (int i = 1; i < NV; ++i) t = join(t, s[i], -kInf);
                if (lanes >= 2) t = join(t, dpp<0xB1>(t.a), dpp<0xB1>(t.b));
                if (lanes >= 4) t = join(t, dpp<0x4E>(t.a), dpp<0x4E>(t.b));
                if (lanes >= 8) t = join(t, dpp<0x141>(t.a), dpp<0x141>(t.b));
                if (lanes >= 16) t = join(t, dpp<0x140>(t.a), dpp<0x140>(t.b));
                mine_score = p.best == 2 && t.b > -kInf ? t.a + t.b : t.a;
                if (e0 < p.n) score32[e0 * p.group_factor >> 20] = mine_score;
                wave_lds_sync();
            } else {
                float* q32 = reinterpret_cast<float*>(q_of);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (e0 + i < p.n) q32[e0 + i] = s[i];
                wave_lds_sync();
                for (int g = l; g < p.groups; g += L) {
                    Best2 t{-kInf, -kInf};
                    for (int e = g * per; e < (g + 1) * per; ++e) t = join(t, q32[e], -kInf);
                    score32[g] = p.best == 2 && t.b > -kInf ? t.a + t.b : t.a;
                }
                wave_lds_sync();
            }
            // a group stays if fewer than top_groups could be before it, and goes if as many
            // surely are
            for (int g = l; g < p.groups; g += L) {
                int could = 0, surely = 0;
                const float v = score32[g];
                for (int h = 0; h < p.groups; ++h) {
                    const float o = score32[h];
                    could += h != g && o >= v - 2.0f * tol;
                    surely += o > v + 2.0f * tol;
                }
                const bool some = v > -kInf;
                stays[g] = some && could < p.top_groups;
                close |= some && could >= p.top_groups && surely < p.top_groups;
            }
            wave_lds_sync();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = e0 + i;
            bool on = there[i] && !bad;
            if (p.groups > 1) on = on && stays[(e < p.n ? e : 0) * p.group_factor >> 20];
            key[i] = on ? (p.bias ? s[i] : x[i]) : -kInf;
        }
        close |= choose<L, NV, float>(key, x, l, p.n, p.k, p.bias ? tol : -1.0f, id, xs);
        if (__ballot(close && ranked && !bad)) {
            // some row of the wavefront is too close to call: scores in fp64
            double q[NV], wide = 1.0;
            if (!p.sigmoid) {
                wide = 0.0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    q[i] = x[i] > -kInf ? exp(double(x[i]) - double(top)) : 0.0;
                    wide += q[i];
                }
                wide = row_add<L>(wide);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                q[i] = p.sigmoid ? 1.0 / (1.0 + exp(-double(x[i]))) : q[i] / wide;
                q[i] = there[i] ? q[i] + double(b[i]) : -double(kInf);
            }
            if (p.groups > 1) {
                wave_lds_sync();
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (e0 + i < p.n) q_of[e0 + i] = q[i];
                wave_lds_sync();
                for (int g = l; g < p.groups; g += L) {
                    double a = -double(kInf), c = -double(kInf);
                    for (int e = g * per; e < (g + 1) * per; ++e) {
                        const double v = q_of[e];
                        c = fmax(c, fmin(a, v));
                        a = fmax(a, v);
                    }
                    score[g] = p.best == 2 && c > -double(kInf) ? a + c : a;
                }
                wave_lds_sync();
                for (int g = l; g < p.groups; g += L) {
                    int before = 0;
                    const double v = score[g];
                    for (int h = 0; h < p.groups; ++h)
                        before += score[h] > v || (score[h] == v && h < g);
                    stays[g] = before < p.top_groups;
                }
                wave_lds_sync();
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = e0 + i;
                bool on = there[i] && !bad;
                if (p.groups > 1) on = on && stays[(e < p.n ? e : 0) * p.group_factor >> 20];
                q[i] = on ? (p.bias ? q[i] : double(x[i])) : -double(kInf);
            }
            wave_lds_sync();
            choose<L, NV, double>(q, x, l, p.n, p.k, -1.0, id, xs);
        }
        wave_lds_sync();
        // weights from the chosen logits
        float high = -kInf;
        if (p.renormalise && !p.sigmoid)
            for (int r = 0; r < p.k; ++r) high = __builtin_fmaxf(high, xs[r]);
        for (int r = l; r < p.k; r += L) {
            const double v = xs[r];
            double w = 0.0;
            if (id[r] < p.n) {
                if (p.sigmoid) w = 1.0 / (1.0 + exp(-v));
                else if (p.renormalise) w = exp(v - double(high));
                else w = exp(v - double(top)) / total;
            }
            share[r] = w;
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
            load_logits<T, NV>(x, l * NV, live ? p.n : 0, s);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (l * NV + i >= p.n) s[i] = -kInf;
                top = __builtin_fmaxf(top, s[i]);
            }
            top = row_max<L>(top);
            total = 0.0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i] = l * NV + i < p.n ? expf(s[i] - top) : 0.0f;
                total += double(s[i]);
            }
            total = row_add<L>(total);
            const float inv = float(1.0 / total);
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] *= inv;
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
        if (live && (l + 1) * NV <= p.n) {
            T packed[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) packed[i] = T(out[i]);
            __builtin_memcpy(p.gx + row * p.n + l * NV, packed, sizeof packed);
        } else if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (l * NV + i < p.n) p.gx[row * p.n + l * NV + i] = T(out[i]);
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
    // exact below 2^10 experts: the factor is less than one part in 2^20 / e too large
    p.group_factor = ((1 << 20) + a.n / a.r.groups - 1) / (a.n / a.r.groups);
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
