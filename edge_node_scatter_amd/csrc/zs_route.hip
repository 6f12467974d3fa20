// Routing of rows to experts and its gradient, gfx950.
//
//   s = softmax(x) or sigmoid(x) of a row, q = s + bias;  of the experts that are there
//   (x and bias above -inf) in the top_groups groups of largest score (the sum of
//   the group's best one or two q) the k of largest q, ties to the lowest index;
//   w_j = a s_ij, or a p_j with p_j = s_ij / sum_l s_il
//
// backward, the choice held fixed, over the slots that hold an expert:
//   renormalised: dx_ij = a p_j (gw_j - m), m = sum_l p_l gw_l, times 1 - s_ij for sigmoid
//   sigmoid:      dx_ij = a gw_j s_ij (1 - s_ij)
//   softmax:      dx_e = a s_e (G_e - m), m = sum_f s_f G_f, G_e the sum of gw over e's slots
// Where one expert has nearly all of a row, G_e and m are nearly the same: subtracted in
// fp32 the rest has no digit left at 18 above the other logits.  Slots' gradients are formed
// in fp64 as (G_e - h) - sum_f s_f (G_f - h), h the G where most of the sum is.
//
// A row lies in the registers of L lanes, NV consecutive experts each.  The choice has to
// be that of fp64 sums (two experts may differ by less than fp32 holds), at the price of
// fp32: fp32 sums pick the groups and some more candidates than there are slots, by
// halving a range of keys and counting; only candidates are ranked in fp64.  Groups that
// fp32 cannot tell, and candidates that may not be all, are settled in fp64 over the whole
// row, which is slow and rare (with random logits a row in a thousand).
//
// Bound by vector instructions, some 520 a row at 256 experts.  Measured on MI355X:
//  - 16384 rows of 256 experts in 8 groups, 8 slots, bf16: 22 us (8.4 MB are read, 1.6
//    written: 2 us at a copy's rate).  All in fp64, a wavefront a row, the largest key
//    by lane reductions: 48 us; fp32 checked by gaps, whole rows anew in fp64: 35
//    (rows that went that way ended 15 us after the rest); 16 lanes a row: 30; 64: 33.
//  - gradients of 8191 rows of 160 experts, 6 slots, fp32: 8.5 us (11 MB), 6.8 with
//    renormalised weights; 65536 rows of 64 experts, one slot: 14 (15 with the same steps in a
//    loop over rows, whose constants took 28 registers and a wavefront a SIMD).
#include "zs_launch.h"
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
    int64_t block0;   // number of the launch's first workgroup
    int n, k, groups, top_groups, best;
    int per_group, group_factor;   // e * group_factor >> 20 is the group of expert e
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
__device__ inline int from_lane(int v) {
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
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
__device__ inline void halves(int v, int& a, int& b) {
    uint32_t x, y;
    halves<WIDE>(uint32_t(v), x, y);
    a = int(x), b = int(y);
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
// fp32 values as integers of the same order (zeros are +0 here): integers are compared
// across lanes without the steps that keep a float's NaN rules.
__device__ inline int key_of(float v) {
    const int b = __builtin_bit_cast(int, v);
    return b ^ (b >> 31 & 0x7fffffff);
}
__device__ inline float value_of(int k) {
    return __builtin_bit_cast(float, k ^ (k >> 31 & 0x7fffffff));
}
template <int L>
__device__ inline int row_max(int v) {
    return over_row<L>(v, [](int a, int b) { return a > b ? a : b; });
}
template <int L>
__device__ inline float row_max(float v) {
    return value_of(row_max<L>(key_of(v)));
}
template <int L>
__device__ inline int row_add(int v) {
    return over_row<L>(v, [](int a, int b) { return a + b; });
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

// e^d for d <= 0, off by less than two ulps: 2^(d log2 e) with what the product's rounding
// and the constant leave out.  Below e^-87 it is 0.
__device__ inline float exp_below(float d) {
    d = __builtin_fmaxf(d, -200.0f);   // the rest of the product stays a number
    const float t = d * 1.44269502162933349609375f;
    const float rest = __builtin_fmaf(d, 1.44269502162933349609375f, -t) +
                       d * 1.925963033500e-8f;
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, rest * 0.693147180559945f, e);
}

// NV values from an address of any alignment; `fill` behind the row's end.
template <typename T, int NV>
__device__ inline void load_values(const T* row, int at, int n, float fill, float (&x)[NV]) {
    if (at + NV <= n) {
        T raw[NV];
        __builtin_memcpy(raw, row + at, sizeof raw);
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = float(raw[i]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = at + i < n ? float(row[at + i]) : fill;
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

// A group's score from its best two.  One expert that is there makes it a group: the sum
// of two that leaves fp32 downwards (biases of the type's lowest value as masks) is the
// lowest value, below every other and beside its like, which fp64 tells apart.
__device__ inline float score_of(Best2 t, int best) {
    const float sum = best == 2 && t.b > -kInf ? t.a + t.b : t.a;
    return t.a > -kInf ? __builtin_fmaxf(sum, -__FLT_MAX__) : -kInf;
}

// A row's part of LDS: all experts' keys (4 bytes each), the candidates' keys and scores
// in fp64 (8 each), the slots' scores (8), the groups' scores in fp32, or in fp64 (8), the
// indices of candidates and slots (4 each) and whether the groups stay (4).
constexpr int kSpare = 8;   // candidates beside the slots
struct RowLds {
    double *key, *chance, *share, *score;
    float* keys;
    int *candidate, *id, *stays;
};
template <int L, int NV>
__host__ __device__ inline int row_bytes(int k, int groups) {
    return (L * NV * 4 + (3 * k + 2 * kSpare + groups) * 8 + (2 * k + kSpare + groups) * 4 + 15) /
           16 * 16;
}
template <int L, int NV>
__device__ inline RowLds row_lds(char* mine, int k, int groups) {
    RowLds r;
    r.keys = reinterpret_cast<float*>(mine);   // on 16 bytes
    r.key = reinterpret_cast<double*>(r.keys + L * NV);
    r.chance = r.key + k + kSpare;
    r.share = r.chance + k + kSpare;
    r.score = r.share + k;
    r.candidate = reinterpret_cast<int*>(r.score + groups);
    r.id = r.candidate + k + kSpare;
    r.stays = r.id + k;
    return r;
}

// Marks the row's largest keys, at least `take` of them and at most `room`: bit i of the
// result is the lane's key[i].  Where equal keys leave no such choice, exactly `take`, of
// the equal ones those of lowest index.  The key they start at is found by halving the
// range between the row's largest and smallest and counting; the middle is taken of the
// values at first, which is quick for values of one size, and then of their bit
// patterns, which ends after 32 steps for any.  take <= have, the keys above -inf, and
// take <= room.  least_marked: no marked key is below it, no other one above it, and none
// at it unless +inf is returned (equal keys were told apart by their index).
template <int L, int NV>
__device__ inline uint32_t mark_largest(const float (&key)[NV], int l, int have, int take, int room,
                                        float& least_marked) {
    float most = key[0], least = key[0] > -kInf ? key[0] : kInf;
#pragma unroll
    for (int i = 1; i < NV; ++i) {
        most = __builtin_fmaxf(most, key[i]);
        least = __builtin_fminf(least, key[i] > -kInf ? key[i] : kInf);
    }
    // at least `take` keys from lo on, fewer from hi on
    int lo = -row_max<L>(-key_of(least)), hi = row_max<L>(key_of(most)) + 1, above = 0;
    bool done = have <= room;
    int bound = done ? lo : hi;   // the marked keys are those from here on ...
    for (int step = 0; __ballot(!done) != 0; ++step) {
        int mid = lo + int((uint32_t(hi) - uint32_t(lo)) >> 1);
        if (step < 8) {   // uniform
            const int m = key_of(0.5f * value_of(lo) + 0.5f * value_of(hi) + 0.0f);
            if (m > lo && m < hi) mid = m;
        }
        const float t = value_of(mid);
        int c = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) c += key[i] >= t;
        c = row_add<L>(c);
        if (done) continue;
        if (uint32_t(hi) - uint32_t(lo) <= 1) done = true;
        else if (c > room) lo = mid;
        else if (c >= take) bound = mid, above = take, done = true;
        else hi = bound = mid, above = c;
    }
    uint32_t mask = 0;
    const float from = value_of(bound);
#pragma unroll
    for (int i = NV - 1; i >= 0; --i) mask = mask + mask + (key[i] >= from ? 1 : 0);
    // ... and as many as are missing of those one below, in the order of their index
    const int missing = have <= room ? 0 : take - above;
    least_marked = missing > 0 ? kInf : from;
    if (__ballot(missing > 0)) {
        const float tie = value_of(lo);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) mine += key[i] == tie;
        int before = mine;   // of lower lanes
#pragma unroll
        for (int d = 1; d < L; d *= 2) {
            const int v = __shfl_up(before, d, L);
            before += l >= d ? v : 0;
        }
        before -= mine;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] == tie && before < missing) ++before, mask |= 1u << i;
    }
    return mask;
}

// An expert's score in fp64.
__device__ inline double score64(double x, bool sigmoid, double top, double total) {
    return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / total;
}

// A softmax's sum in fp64 (lean in registers, as few rows need it).
template <typename T, int L>
__device__ inline double total64(const T* logits, int n, double top, int l) {
    double total = 0.0;
#pragma unroll 1
    for (int e = l; e < n; e += L) {
        const double v = float(logits[e]);
        total += v > -double(kInf) ? exp(v - top) : 0.0;
    }
    return row_add<L>(total);
}

// Which groups stay, from scores in fp64: for rows that fp32 cannot tell.
template <typename T, int L>
__device__ inline void groups64(const RouteParams<T>& p, const T* logits, int n, float top, int l,
                                const RowLds& r) {
    constexpr double none = -double(kInf);
    const double total = p.sigmoid ? 1.0 : total64<T, L>(logits, n, top, l);
    // a group at a time, as many lanes as there are at its experts
    for (int g = 0; g < p.groups; ++g) {
        double a = none, b = none;
#pragma unroll 1
        for (int i = l; i < p.per_group; i += L) {
            const int e = g * p.per_group + i;
            const double x = e < n ? double(float(logits[e])) : none;
            const double bias = p.bias ? double(p.bias[e]) : 0.0;
            const double q = x > none && bias > none
                                 ? score64(x, p.sigmoid, top, total) + bias : none;
            b = fmax(b, fmin(a, q));
            a = fmax(a, q);
        }
        const double most = over_row<L>(a, [](double x, double y) { return x > y ? x : y; });
        // the second is the largest of what is left once one lane has given its largest
        const uint64_t who = row_ballot<L>(a == most);
        const double rest = who && l == __builtin_ctzll(who) ? b : a;
        const double next = over_row<L>(rest, [](double x, double y) { return x > y ? x : y; });
        if (l == 0) r.score[g] = p.best == 2 && next > none ? most + next : most;
    }
    wave_lds_sync();
    for (int g = l; g < p.groups; g += L) {
        int before = 0;
        const double v = r.score[g];
        for (int h = 0; h < p.groups; ++h)
            before += r.score[h] > v || (r.score[h] == v && h < g);
        r.stays[g] = v > none && before < p.top_groups;
    }
    wave_lds_sync();
}

// The k experts of largest sum in fp64, by rounds over all of them: for rows with more
// experts too close to call than there are candidates (as with equal logits and no bias
// yet).  Rows that only share the wavefront with one keep theirs.
template <typename T, int L>
__device__ inline void choose64(const RouteParams<T>& p, const T* logits, int n, float top, int l,
                                const RowLds& r, bool mine) {
    constexpr double none = -double(kInf);
    const double total = p.sigmoid ? 1.0 : total64<T, L>(logits, n, top, l);
    double last = double(kInf);   // the sum and index of the round before
    int last_at = -1;
    for (int j = 0; j < p.k; ++j) {
        double best = none;
        int at = p.n;
#pragma unroll 1
        for (int e = l; e < n; e += L) {
            const double x = float(logits[e]), bias = double(p.bias[e]);
            if (!(x > none && bias > none) || !(r.keys[e] > -kInf)) continue;
            const double q = score64(x, p.sigmoid, top, total) + bias;
            const bool left = q < last || (q == last && e > last_at);
            if (left && q > best) best = q, at = e;   // (ties: the lane's lowest)
        }
        const double m = over_row<L>(best, [](double x, double y) { return x > y ? x : y; });
        last_at = -row_max<L>(best == m && m > none ? -at : -p.n);
        last = m;
        if (mine && l == 0) r.id[j] = last_at;
        if (last_at == p.n) last = none;
    }
    wave_lds_sync();
    for (int j = l; mine && j < p.k; j += L)
        r.share[j] = r.id[j] < p.n ? score64(float(logits[r.id[j]]), p.sigmoid, top, total) : 0.0;
    wave_lds_sync();
}

template <typename T, int L, int NV>
__global__ __launch_bounds__(kThreads) void zs_route_kernel(const RouteParams<T> p) {
    extern __shared__ __align__(16) char lds[];
    const int l = threadIdx.x % L, slot = threadIdx.x / L, e0 = l * NV;
    const RowLds r = row_lds<L, NV>(lds + slot * row_bytes<L, NV>(p.k, p.groups), p.k, p.groups);
    float* group_score = reinterpret_cast<float*>(r.score);
    const bool ranked = p.bias || p.groups > 1;   // by more than the logits
    // lanes that hold a group, if whole lanes do and DPP joins them
    const int lanes = p.per_group / NV;
    const bool joined =
        p.per_group % NV == 0 && lanes <= (L < 16 ? L : 16) && (lanes & (lanes - 1)) == 0;
    float b[NV], bias_size = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) b[i] = 0.0f;
    if (p.bias) {
        load_values<float, NV>(p.bias, e0, p.n, 0.0f, b);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // NaN is -inf from here on: a minimum with NaN is the other operand, so that a
            // group's best would be its second best too
            b[i] = b[i] > -kInf ? b[i] : -kInf;
            bias_size = __builtin_fmaxf(bias_size, b[i] > -kInf ? __builtin_fabsf(b[i]) : 0.0f);
        }
        bias_size = row_max<L>(bias_size);
    }
    const int64_t row = (p.block0 + blockIdx.x) * (kThreads / L) + slot;
    const bool live = row < p.n_rows;
    const int n = live ? p.n : 0;
    const T* logits = p.x + row * p.ldx;
    float x[NV];
    bool bad = false;
    load_values<T, NV>(logits, e0, n, -kInf, x);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        x[i] += 0.0f;   // -0 is +0, and no signalling NaN
        bad |= x[i] != x[i];
    }
    float top = -kInf;
    if (!p.sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; ++i) top = __builtin_fmaxf(top, x[i]);
        top = row_max<L>(top);
        bad |= top == kInf;
    }
    bad = row_ballot<L>(bad) != 0;
    // Sums of score and bias in fp32, and how far two of them may lie apart that fp64
    // might order otherwise.  A score is off by at most 10 units of 2^-24 of the row's
    // largest (softmax: two ulps of the exponential, the rounding of its argument d, of
    // which e^-d d <= 0.37 counts, 4 for the sum and 3 for two products) or of 1
    // (sigmoid: less), the sum by half an ulp; two of them, and some to spare.
    float s[NV], most = 1.0f;
    double total = 1.0;
    if (!p.sigmoid && (ranked || !p.renormalise)) {
        total = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            s[i] = x[i] > -kInf ? exp_below(x[i] - top) : 0.0f;
            total += double(s[i]);
        }
        total = row_add<L>(total);
        most = total > 0.0 ? 1.0f / float(total) : 1.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] *= most;
    } else if (ranked) {
        // 2^(-x log2 e); what overflows or underflows in it leaves the score 0 or 1
#pragma unroll
        for (int i = 0; i < NV; ++i)
            s[i] = __builtin_amdgcn_rcpf(1.0f +
                                         __builtin_amdgcn_exp2f(x[i] * -1.44269504088896341f));
    }
    const float tol = most * 0x1p-19f + (most + bias_size) * 0x1p-22f;
    if (ranked)
        // -inf where the bias is
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = x[i] > -kInf ? s[i] + b[i] : -kInf;
    bool here = !bad;   // the lane's group stays, if it holds one
    if (p.groups > 1) {
        if (joined) {
            Best2 t{-kInf, -kInf};
#pragma unroll
            for (int i = 0; i < NV; ++i) t = join(t, s[i], -kInf);
            if (lanes >= 2) t = join(t, dpp<0xB1>(t.a), dpp<0xB1>(t.b));
            if (lanes >= 4) t = join(t, dpp<0x4E>(t.a), dpp<0x4E>(t.b));
            if (lanes >= 8) t = join(t, dpp<0x141>(t.a), dpp<0x141>(t.b));
            if (lanes >= 16) t = join(t, dpp<0x140>(t.a), dpp<0x140>(t.b));
            if (e0 < p.n)
                group_score[e0 * p.group_factor >> 20] = score_of(t, p.best);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) r.keys[e0 + i] = s[i];
            wave_lds_sync();
            for (int g = l; g < p.groups; g += L) {
                Best2 t{-kInf, -kInf};
                for (int e = g * p.per_group; e < (g + 1) * p.per_group; ++e)
                    t = join(t, r.keys[e], -kInf);
                group_score[g] = score_of(t, p.best);
            }
        }
        wave_lds_sync();
        // a group stays if fewer than top_groups could be before it, and goes if as many
        // surely are
        bool close = false;
        for (int g = l; g < p.groups; g += L) {
            int could = 0, surely = 0;
            const float v = group_score[g];
            const float low = v - 2.0f * tol, high = v + 2.0f * tol;
            for (int h = 0; h < p.groups; ++h) {
                const float o = group_score[h];
                could += o >= low;   // the group itself too
                surely += o > high;
            }
            const bool some = v > -kInf;
            r.stays[g] = some && could <= p.top_groups;
            // (a bias of +inf leaves no bound)
            close |= some && !(could <= p.top_groups || surely >= p.top_groups);
            close |= !(tol < kInf);
        }
        wave_lds_sync();
        if (__ballot(close && !bad)) groups64<T, L>(p, logits, n, top, l, r);
        if (joined) here = here && e0 < p.n && r.stays[e0 * p.group_factor >> 20];
    }
    // the keys: sums, or logits without a bias
    int have = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        bool on = here;
        if (p.groups > 1) {
            if (!joined)
                on = on && r.stays[(e0 + i < p.n ? e0 + i : 0) * p.group_factor >> 20];
            if (!p.bias) s[i] = s[i] > -kInf ? x[i] : -kInf;
        } else if (!p.bias) {
            s[i] = x[i];
        }
        s[i] = on ? s[i] : -kInf;
        have += s[i] > -kInf;
    }
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < NV; ++i) r.keys[e0 + i] = s[i];
    have = row_add<L>(have);
    // Candidates: with a bias two more than the slots at least, so that the first that is not
    // one lies clearly behind the last slot.
    const int room = p.k + kSpare, want = p.bias ? p.k + 2 : p.k;
    float least;
    uint32_t mask = mark_largest<L, NV>(s, l, have, have < want ? have : want, room, least);
    int at = __builtin_popcount(mask);
    const int mine = at;
#pragma unroll
    for (int d = 1; d < L; d *= 2) {
        const int v = __shfl_up(at, d, L);
        at += l >= d ? v : 0;
    }
    const int marked = __shfl(at, L - 1, L);
    at -= mine;
    for (; mask != 0; mask &= mask - 1) r.candidate[at++] = e0 + __builtin_ctz(mask);
    wave_lds_sync();
    // Their keys in fp64, and their places among each other.  In a softmax with a bias fp64
    // scores need the sum in fp64 as well: where two lie close to each other, once more with
    // that.  (The row's own decision: its weights have the same bits beside any rows.)
    bool unsettled = false;   // what is no candidate may belong to the slots
    for (int pass = 0;; ++pass) {
        for (int i = l; i < marked; i += L) {
            const int e = r.candidate[i];
            double v = r.keys[e];
            if (p.bias) {
                v = score64(float(logits[e]), p.sigmoid, top, total);
                r.chance[i] = v;
                v += double(p.bias[e]);
            }
            r.key[i] = v;
        }
        wave_lds_sync();
        bool close = false;
        unsettled = false;
        for (int i = l; i < marked; i += L) {
            const double own = r.key[i];
            int rank = 0;   // (candidates lie in the order of their index)
#pragma unroll 4
            for (int j = 0; j < marked; ++j) {
                const double o = r.key[j];
                rank += o > own || (o == own && j < i);
            }
            if (p.bias) {
                if (pass == 0 && !p.sigmoid)
                    for (int j = 0; j < marked; ++j)
                        close |= j != i && __builtin_fabs(r.key[j] - own) <= double(tol);
                unsettled |= rank == p.k - 1 && marked < have &&
                             !(own >= double(least) + double(tol));
                if (rank < p.k) r.share[rank] = r.chance[i];
            }
            if (rank < p.k) r.id[rank] = r.candidate[i];
        }
        if (pass == 1 || !p.bias || p.sigmoid || __ballot(close) == 0) break;
        const double exact = total64<T, L>(logits, n, top, l);
        if (row_ballot<L>(close)) total = exact;
        wave_lds_sync();
    }
    for (int j = marked + l; j < p.k; j += L) r.id[j] = p.n;
    wave_lds_sync();
    if (__ballot(unsettled))
        choose64<T, L>(p, logits, n, top, l, r, row_ballot<L>(unsettled) != 0);
    // the slots' scores or, renormalised in a softmax, exponentials above the largest chosen
    if (!p.bias || (p.renormalise && !p.sigmoid)) {
        float high = top;
        if (p.renormalise && !p.sigmoid) {
            high = -kInf;
            for (int j = l; j < p.k; j += L)
                if (r.id[j] < p.n) high = __builtin_fmaxf(high, float(logits[r.id[j]]));
            high = row_max<L>(high);
        }
        const double whole = p.renormalise ? 1.0 : total;
        for (int j = l; j < p.k; j += L)
            if (r.id[j] < p.n)
                r.share[j] = score64(float(logits[r.id[j]]), p.sigmoid, high, whole);
        wave_lds_sync();
    }
    double sum = 1.0;
    if (p.renormalise) {
        sum = 0.0;
        for (int j = 0; j < p.k; ++j)
            if (r.id[j] < p.n) sum += r.share[j];
    }
    for (int j = l; live && j < p.k; j += L) {
        const double v = r.id[j] < p.n && sum > 0.0 ? r.share[j] / sum : 0.0;
        p.weight[row * p.k + j] = bad ? __builtin_nanf("") : float(double(p.scale) * v);
        p.expert[row * p.k + j] = r.id[j];
    }
}

// Bytes of LDS of a row in the backward: a slot's share, its gradient and that of its
// expert's slots together (8 each), its index (4).
__host__ __device__ inline int back_bytes(int k) { return k * 32; }

template <typename T, int L, int NV>
__global__ __launch_bounds__(kThreads) void zs_route_bwd_kernel(const RouteParams<T> p) {
    extern __shared__ char lds[];
    const int l = threadIdx.x % L, slot = threadIdx.x / L;
    double* share = reinterpret_cast<double*>(lds + slot * back_bytes(p.k));
    double* grad = share + p.k;
    double* joint = grad + p.k;
    int* id = reinterpret_cast<int*>(joint + p.k);
    const bool full = !p.sigmoid && !p.renormalise;   // every logit has a part in the weights
    const int64_t row = (p.block0 + blockIdx.x) * (kThreads / L) + slot;
    const bool live = row < p.n_rows;
    const T* x = p.x + row * p.ldx;
    float s[NV];
    float top = -kInf;
    if (full) {
        load_values<T, NV>(x, l * NV, live ? p.n : 0, -kInf, s);
#pragma unroll
        for (int i = 0; i < NV; ++i) top = __builtin_fmaxf(top, s[i]);
        top = row_max<L>(top);
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = s[i] > -kInf ? exp_below(s[i] - top) : 0.0f;
    }
    // the slots' logits, the largest of the lane's with its gradient, and the gradients
    float own = -kInf;
    double near = 0.0;
    int live_slots = 0;
    for (int r = l; r < p.k; r += L) {
        const int64_t e = live ? p.chosen[row * p.k + r] : -1;
        const bool in = e >= 0 && e < p.n;
        const float v = in ? float(x[e]) : -kInf;
        const double g = in ? double(p.gw[row * p.k + r]) * double(p.scale) : 0.0;
        id[r] = in ? int(e) : -1, share[r] = v, grad[r] = g;
        if (v > own) own = v, near = g;
        live_slots += in;
    }
    // of all of the row, or of its slots
    const float high = full ? top : row_max<L>(own);
    const bool any = row_ballot<L>(live_slots > 0) != 0;
    wave_lds_sync();
    if (full) {
        uint32_t chosen = 0;   // bit i: some slot holds the lane's expert i
        for (int r = 0; r < p.k; ++r) {
            const unsigned at = unsigned(id[r] - l * NV);
            chosen |= (at < NV ? 1u : 0u) << (at & 31);
        }
        // theirs are formed in fp64
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = chosen >> i & 1 ? 0.0f : s[i];
        // an expert in several slots: the first of them takes all their gradients
        if (p.k > 1 &&
            __ballot(row_add<L>(__builtin_popcount(chosen) - live_slots) != 0) != 0) {
            for (int r = l; r < p.k; r += L) {
                double g = 0.0;
                bool first = true;
                for (int q = 0; q < p.k; ++q)
                    if (id[q] == id[r]) g += grad[q], first &= q >= r;
                joint[r] = first ? g : 0.0;
                if (share[r] == double(high)) near = g;
                if (!first) share[r] = -double(kInf);
            }
            wave_lds_sync();
            for (int r = l; r < p.k; r += L) grad[r] = joint[r];
        }
    }
    // the gradients' mean is formed as what lies between it and the gradient where most of
    // the sum is: that of the slot of largest logit, or 0 if that expert is in no slot
    const uint64_t who = row_ballot<L>(own == high);
    near = __shfl(near, who ? __builtin_ctzll(who) : 0, L);
    if (who == 0) near = 0.0;
    double sum = 0.0, between = 0.0, inv = 1.0;
    if (full) {
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += double(s[i]);
        between = -near * sum;
    }
    for (int r = l; r < p.k; r += L) {
        const double v = share[r];
        double w = 0.0;
        if (id[r] >= 0) {
            if (p.sigmoid) w = 1.0 / (1.0 + exp(-v));
            else w = exp(v - double(high));
        }
        share[r] = w;
        sum += w;
        between += w * (grad[r] - near);
    }
    if (p.renormalise || full) {
        sum = row_add<L>(sum);
        if (!(sum > 0.0)) sum = 1.0;   // all shares are 0
        between = row_add<L>(between);
        if (p.sigmoid) {   // (the inverse of a sum of tiny scores is above fp64's range)
            between /= sum;
        } else {
            inv = 1.0 / sum;
            between *= inv;
        }
    }
    for (int r = l; r < p.k; r += L) {
        const double w = share[r], g = grad[r], rest = (g - near) - between;
        if (p.sigmoid) grad[r] = (p.renormalise ? w / sum * rest : g * w) * (1.0 - w);
        else grad[r] = w * inv * rest;
    }
    wave_lds_sync();
    float out[NV];
    const float each = -float((near + between) * inv);
#pragma unroll
    for (int i = 0; i < NV; ++i) out[i] = full && any ? s[i] * each : 0.0f;
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
}

template <typename T, int L, int NV>
hipError_t run(const RouteArgs& a, bool backward, hipStream_t stream) {
    RouteParams<T> p{};
    p.x = static_cast<const T*>(a.x), p.bias = a.bias, p.ldx = a.ldx, p.n_rows = a.n_rows;
    p.n = a.n, p.k = a.r.k, p.groups = a.r.groups, p.top_groups = a.r.top_groups;
    p.best = a.r.best, p.sigmoid = a.r.sigmoid != 0, p.renormalise = a.r.renormalise != 0;
    p.per_group = a.n / a.r.groups;
    // exact below 2^10 experts: the factor is less than one part in 2^20 / e too large
    p.group_factor = ((1 << 20) + p.per_group - 1) / p.per_group;
    p.scale = a.r.scale, p.weight = a.weight, p.expert = a.expert;
    p.gw = a.gw, p.chosen = a.chosen, p.gx = static_cast<T*>(a.gx);
    constexpr int rows = kThreads / L;
    const int64_t want = (a.n_rows + rows - 1) / rows;
    // (no loop over rows in the kernels: what the compiler took out of it cost as many registers
    // again as the rows' own values)
    return launch_ranges(want, kThreads, [&](int64_t first, int64_t count) {
        p.block0 = first;
        if (backward)
            zs_route_bwd_kernel<T, L, NV>
                <<<unsigned(count), kThreads, size_t(rows) * back_bytes(p.k), stream>>>(p);
        else
            zs_route_kernel<T, L, NV>
                <<<unsigned(count), kThreads, size_t(rows) * row_bytes<L, NV>(p.k, p.groups),
                   stream>>>(p);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t dispatch(const RouteArgs& a, bool backward, hipStream_t stream) {
    if (a.n <= 8) return run<T, 8, 1>(a, backward, stream);
    if (a.n <= 32) return run<T, 8, 4>(a, backward, stream);
    if (a.n <= 64) return run<T, 16, 4>(a, backward, stream);
    if (a.n <= 128) return run<T, 16, 8>(a, backward, stream);
    if (a.n <= 256) return run<T, 32, 8>(a, backward, stream);
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
