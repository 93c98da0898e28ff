// The router's choice and its gradient.
//
// Choice.  An expert's choice value c is its logit, or its score plus bias
// where a bias or groups take part; a row's k largest are chosen, the lowest
// index first among equals.  A bf16 logit and the index make one integer of 32
// bits.  Other choice values are kept as a binary64 number whose 12 lowest
// bits hold the index (turned round for c >= 0, so that a lower index is
// larger): comparing two keys compares values, then indexes, in one
// instruction, and no two keys are equal.  A binary32 logit has those bits
// free; scores are computed in 64 bits and rounded to 41, so that values which
// are equal but for roundings tie (as the sigmoids of 1 and -1 and twice that
// of 0, in groups).
//
// A row belongs to L lanes, P experts each.  Every lane sorts its keys; then k
// times the largest of the lanes' first ones is taken, and its lane moves up.
//
// Weights.  With m the largest chosen logit:
//     softmax, normalised   exp(z - m) / sum over the chosen
//     softmax               exp(z - max) / sum over all
//     sigmoid, normalised   r / sum of the chosen r,
//                           r = exp(min(z, 0) - min(m, 0)) / (1 + exp(-|z|))
//     sigmoid               exp(min(z, 0)) / (1 + exp(-|z|))
// r is the score over a common factor, so that scores that vanish still have
// their shares.
//
// Gradient, with w = scale * s the weights, g their gradient times scale:
//     normalised            dz = s (g - sum_i g_i s_i), sigmoid: times 1 - score
//     softmax               dz = p ([chosen] g - sum_i g_i p_i), all experts
//     sigmoid               dz = g s (1 - s)
//
// What bounds it.  131072 rows of 256 bf16 logits, top-8: 32 us forward (75 MB,
// 2.4 TB/s), instructions: about a third each for the sort, the k rounds, and the
// exponentials with the keys; 28 us backward (142 MB, 5 TB/s).  128 rows
// with bias and groups: 6.5 us, latency of dependent lane exchanges (13 with 16
// lanes a row).  The compiler's accesses by index for lists that move up took
// 343 us forward, binary64 keys for bf16 logits 44.
#include <type_traits>

#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kRouterThreads = 256;
constexpr int kMaxGroups = 64;
constexpr int kMaxSlots = 32;

template <int CTRL>
__device__ inline double dpp64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// As row_reduce (experts_common.h), of binary64 values over L = 16 or 64 lanes.
template <int L, class OP>
__device__ inline double row_reduce64(double v, OP op) {
    static_assert(L == 16 || L == 64, "lanes of a row");
    v = op(v, dpp64<0xB1>(v));
    v = op(v, dpp64<0x4E>(v));
    v = op(v, dpp64<0x141>(v));
    v = op(v, dpp64<0x140>(v));
    if (L > 16) {
        uint64_t b = __builtin_bit_cast(uint64_t, v);
        auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
        auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
        v = op(__builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]),
               __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]));
        b = __builtin_bit_cast(uint64_t, v);
        lo = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
        hi = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
        v = op(__builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]),
               __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]));
    }
    return v;
}
// v_max_f64 / v_min_f64 of values that are no NaN.
__device__ inline double max64(double a, double b) { return __builtin_fmax(a, b); }
__device__ inline double min64(double a, double b) { return __builtin_fmin(a, b); }
template <int L>
__device__ inline double lanes_max64(double v) {
    return row_reduce64<L>(v, [](double x, double y) { return max64(x, y); });
}
template <int L>
__device__ inline double lanes_sum64(double v) {
    return row_reduce64<L>(v, [](double x, double y) { return x + y; });
}

// exp(v) for v <= 0 to about 2^-45: 2^n times the series of the rest, |rest| <
// 0.35, to the 11th power (the 12th is 6e-15).  Zero below -700.
__device__ inline double exp64(double u) {
    const double v = max64(u, -700.0);
    const double n = __builtin_rint(v * 0x1.71547652b82fep+0);
    double r = __builtin_fma(n, -0x1.62e42fefa39efp-1, v);
    r = __builtin_fma(n, -0x1.abc9e3b39803fp-56, r);
    double p = 1.0 / 39916800.0;
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return u < -700.0 ? 0.0 : __builtin_ldexp(p, (int)n);
}

// 1 / v for v in [1, 2^1000]
__device__ inline double rcp64(double v) {
    double r = __builtin_amdgcn_rcp(v);
    r = __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
}

// exp(v) for v <= 0 to about a step of binary32: as 2^h (1 + l ln 2), h + l =
// v / ln 2.  Zero below -87, where 2^h leaves the normal range.
__device__ inline float exp32(float v) {
    const float x = fmaxf(v, -87.0f);
    const float h = x * 0x1.715476p+0f;
    float l = __builtin_fmaf(x, 0x1.715476p+0f, -h);
    l = __builtin_fmaf(x, 0x1.4ae0c0p-26f, l);
    const float p = __builtin_amdgcn_exp2f(h);
    const float e = __builtin_fmaf(p, l * 0x1.62e430p-1f, p);
    return v < -87.0f ? 0.0f : e;
}

// Keys: value and index as one number that orders by value, then by the lower
// index.  No two of a row's experts have the same.
struct Key64 {
    using type = double;
    static constexpr double kNone = -__builtin_huge_val();  // no choice
    // c to the nearest of 41 bits; infinity as 2^200, which leaves room for the
    // index.  Only values above kNone.
    static __device__ inline double make(double c, int e) {
        const uint64_t b = __builtin_bit_cast(uint64_t, min64(c, 0x1p200) + 0.0) + 2048u;  // -0 becomes 0
        const uint64_t at = (int64_t)b < 0 ? (uint64_t)e : (uint64_t)(4095 - e);
        return __builtin_bit_cast(double, (b & ~4095ull) | at);
    }
    static __device__ inline int index(double key) {
        const uint64_t b = __builtin_bit_cast(uint64_t, key);
        const int low = (int)(b & 4095u);
        return (int64_t)b < 0 ? low : 4095 - low;
    }
    static __device__ inline double value(double key) {
        return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~4095ull);
    }
    static __device__ inline double larger(double a, double b) { return max64(a, b); }
    static __device__ inline double smaller(double a, double b) { return min64(a, b); }
    template <int L>
    static __device__ inline double largest(double v) { return lanes_max64<L>(v); }
    // a where the mask is all ones, b where it is zero.  (The compiler would turn
    // a choice between neighbours of an array into an access by index.)
    static __device__ inline double pick(uint32_t mask, double a, double b) {
        const uint64_t x = __builtin_bit_cast(uint64_t, a), y = __builtin_bit_cast(uint64_t, b);
        const uint32_t lo = ((uint32_t)x & mask) | ((uint32_t)y & ~mask);
        const uint32_t hi = ((uint32_t)(x >> 32) & mask) | ((uint32_t)(y >> 32) & ~mask);
        return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    }
};
// The bits of a bf16 logit, turned so that they order as integers, with the index
// in the lowest 12.  The 4 above those are zeros, or ones where the bits are
// turned, but for the largest binary32 number: that stands for +inf and has
// to be above the largest bf16 one, which they tell it from.
struct Key32 {
    using type = int32_t;
    static constexpr int32_t kNone = (int32_t)0x807FFFFF;  // the largest key of -inf
    static __device__ inline int32_t make(float z, int e) {
        const int32_t b = __float_as_int(z + 0.0f);  // -0 becomes 0
        return ((b ^ ((b >> 31) & 0x7FFFFFFF)) & ~4095) | (4095 - e);
    }
    static __device__ inline int index(int32_t key) { return 4095 - (key & 4095); }
    static __device__ inline int32_t larger(int32_t a, int32_t b) { return max(a, b); }
    static __device__ inline int32_t smaller(int32_t a, int32_t b) { return min(a, b); }
    template <int L>
    static __device__ inline int32_t largest(int32_t v) {
        auto moved = [](int32_t x, auto ctrl) {
            return __builtin_amdgcn_update_dpp(0, x, decltype(ctrl)::value, 0xF, 0xF, true);
        };
        v = max(v, moved(v, std::integral_constant<int, 0xB1>{}));
        v = max(v, moved(v, std::integral_constant<int, 0x4E>{}));
        v = max(v, moved(v, std::integral_constant<int, 0x141>{}));
        v = max(v, moved(v, std::integral_constant<int, 0x140>{}));
        if (L > 16) {
            auto r = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
            v = max((int32_t)r[0], (int32_t)r[1]);
            r = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
            v = max((int32_t)r[0], (int32_t)r[1]);
        }
        return v;
    }
    static __device__ inline int32_t pick(uint32_t mask, int32_t a, int32_t b) {
        return (int32_t)(((uint32_t)a & mask) | ((uint32_t)b & ~mask));
    }
};

// Descending, by Batcher's odd-even merge network.
template <class K, int N>
__device__ inline void sort_keys(typename K::type v[N]) {
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const auto x = v[i + j], y = v[i + j + q];
                        v[i + j] = K::larger(x, y);
                        v[i + j + q] = K::smaller(x, y);
                    }
}

template <bool BF16>
__device__ inline float raw_logit(const void* logits, size_t at) {
    return BF16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(logits)[at] << 16)
                : reinterpret_cast<const float*>(logits)[at];
}
// +inf counts as the largest finite number, so that differences are numbers;
// NaN as -inf, which takes no part (the larger of NaN and a number is the number).
__device__ inline float tame(float v) { return fminf(fmaxf(v, -INFINITY), 0x1.fffffep+127f); }

// Lane l's logits of a row: experts (c * L + l) * V .. + V - 1 of chunk c, V
// at a time; -inf past the last expert.
template <int P>
constexpr int piece() { return P < 8 ? P : 8; }
template <int L, int P>
__device__ inline int expert_of(int l, int i) {
    constexpr int V = piece<P>();
    return (i / V * L + l) * V + i % V;
}

template <int L, int P, bool BF16>
__device__ inline void load_row(const RouterArgs& a, size_t row, int l, float z[P]) {
    constexpr int V = piece<P>();
#pragma unroll
    for (int c = 0; c < P / V; ++c) {
        const int e0 = (c * L + l) * V;
        if (a.vec) {
            const size_t at = row * a.E + min(e0, a.E - V);
            if constexpr (BF16) {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(a.logits) + at);
                uint32_t w[V / 2];
                if constexpr (V == 8) {
                    const v4u x = *reinterpret_cast<const v4u*>(p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = x[i];
                } else {
                    const v2i x = *reinterpret_cast<const v2i*>(p);
                    w[0] = (uint32_t)x[0];
                    w[1] = (uint32_t)x[1];
                }
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    z[c * V + 2 * i] = bf16_low(w[i]);
                    z[c * V + 2 * i + 1] = bf16_high(w[i]);
                }
            } else {
#pragma unroll
                for (int h = 0; h < V / 4; ++h) {
                    const v4f x = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(a.logits) + at + 4 * h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[c * V + 4 * h + i] = x[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) z[c * V + i] = raw_logit<BF16>(a.logits, row * a.E + min(e0 + i, a.E - 1));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) z[c * V + i] = tame(z[c * V + i]);
    }
    if (a.E == L * P) return;  // no compare per expert (with signed keys: 37 us forward -> 33)
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (expert_of<L, P>(l, i) >= a.E) z[i] = -INFINITY;
}

// Scores over the chosen ones' common factor, and what divides them.  m is the
// largest logit among those that count.  (The difference is rounded: a score far
// below the largest is off by |z - m| half steps, at most 87.)
__device__ inline float part(bool sigmoid, float z, float m) {
    if (!sigmoid) return exp32(z - m);
    return exp32(fminf(z, 0.0f) - fminf(m, 0.0f)) / (1.0f + exp32(-fabsf(z)));
}

// exp(v) for v <= 0, for sums: off by |v| steps, which the terms' own size
// makes up for.
__device__ inline float exp_term(float v) { return __builtin_amdgcn_exp2f(v * 0x1.715476p+0f); }

// Choice values from scores, in 64 bits.  *sum is the softmax's sum.
template <int L, int P>
__device__ inline void score_keys(const RouterArgs& a, int l, const float z[P], float top, double key[P], float* sum) {
    double total = 1.0;
    if (!a.sigmoid) {
        total = 0.0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            key[i] = exp64((double)z[i] - (double)top);
            total += key[i];
        }
        total = lanes_sum64<L>(total);
        *sum = (float)total;
        total = rcp64(total);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int e = expert_of<L, P>(l, i);
        double c;
        if (a.sigmoid) {
            const double zd = (double)z[i];
            const double x = exp64(-__builtin_fabs(zd));
            c = (zd < 0.0 ? x : 1.0) * rcp64(1.0 + x);
        } else {
            c = key[i] * total;
        }
        if (a.bias) c += (double)a.bias[min(e, a.E - 1)];
        // -inf and NaN, also from the bias, are no choice
        key[i] = z[i] > -INFINITY && c > Key64::kNone ? Key64::make(c, e) : Key64::kNone;
    }
}

// Takes away the experts of groups that are not among the best.  A group's
// experts, in LDS, belong to a.group_lanes neighbouring lanes.
template <int L, int P>
__device__ inline void keep_groups(const RouterArgs& a, int l, double* mine, double key[P]) {
    constexpr double kNone = Key64::kNone;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int e = expert_of<L, P>(l, i);
        if (e < a.E) mine[e] = key[i];
    }
    __syncthreads();
    constexpr int kG = kMaxGroups / L;  // passes over the groups, where each has one lane
    const int at_once = L / a.group_lanes;
    const int sub = l % a.group_lanes;
    double group[kG];
#pragma unroll
    for (int h = 0; h < kG; ++h) {
        const int g = h * at_once + l / a.group_lanes;
        double first = kNone, second = kNone;
        if (g < a.groups)
            for (int i = sub; i < a.per_group; i += a.group_lanes) {
                const double v = mine[g * a.per_group + i];
                second = max64(second, min64(first, v));
                first = max64(first, v);
            }
        for (int d = 1; d < a.group_lanes; d <<= 1) {
            const double f = __shfl_xor(first, d), s = __shfl_xor(second, d);
            second = max64(min64(first, f), max64(second, s));
            first = max64(first, f);
        }
        group[h] = kNone;
        if (first > kNone && sub == 0) {
            double v = Key64::value(first);
            if (a.group_best > 1 && second > kNone) v += Key64::value(second);
            group[h] = Key64::make(v, g);
        }
    }
    uint64_t kept = 0;
    for (int j = 0; j < a.topk_groups; ++j) {
        double best = group[0];
#pragma unroll
        for (int h = 1; h < kG; ++h) best = max64(best, group[h]);
        best = lanes_max64<L>(best);
        if (best > kNone) kept |= 1ull << Key64::index(best);
#pragma unroll
        for (int h = 0; h < kG; ++h) group[h] = group[h] == best ? kNone : group[h];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int e = min(expert_of<L, P>(l, i), a.E - 1);
        if (!(kept >> (e / a.per_group) & 1)) key[i] = kNone;
    }
}

// The k largest of a row's lanes' sorted keys, slot h * L + l in slot[h] of lane
// l.  D: entries of a lane that can be among them.
template <class K, int L, int P, int D>
__device__ inline void take(int k, int l, typename K::type key[P], typename K::type slot[(kMaxSlots + L - 1) / L]) {
    for (int j = 0; j < k; ++j) {
        const auto best = K::template largest<L>(key[0]);
#pragma unroll
        for (int h = 0; h < (kMaxSlots + L - 1) / L; ++h) slot[h] = j == h * L + l ? best : slot[h];
        const uint32_t won = key[0] == best ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int i = 0; i + 1 < D; ++i) key[i] = K::pick(won, key[i + 1], key[i]);
        key[D - 1] = K::pick(won, K::kNone, key[D - 1]);
    }
}

// K: Key64, or Key32 for the choice by bf16 logits.
template <class K, int L, int P, bool BF16>
__global__ __launch_bounds__(kRouterThreads) void moedisp_router(RouterArgs a) {
    constexpr int kRows = kRouterThreads / L;
    constexpr int kSlots = (kMaxSlots + L - 1) / L;  // slots of a lane
    constexpr bool k64 = std::is_same<K, Key64>::value;
    extern __shared__ __align__(16) double s_keys[];  // groups: [kRows][E]
    const int l = threadIdx.x % L;
    const long long at = (long long)blockIdx.x * kRows + threadIdx.x / L;
    const bool on = at < a.T && (a.live == nullptr || a.live[at < a.T ? at : 0] != 0);
    const size_t row = at < a.T ? (size_t)at : 0;

    float z[P];
    load_row<L, P, BF16>(a, row, l, z);
    const bool by_score = k64 && (a.bias != nullptr || a.groups > 1);
    float top = 0.0f, sum = 1.0f;  // softmax: the row's largest logit, the sum of exp(z - top)
    if (!a.sigmoid && (by_score || !a.normalise)) {
        top = z[0];
#pragma unroll
        for (int i = 1; i < P; ++i) top = fmaxf(top, z[i]);
        top = lanes_max<L>(top);
        if (!by_score) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) sum += exp_term(z[i] - top);
            sum = lanes_sum<L>(sum);
        }
    }
    typename K::type key[P];
    if constexpr (k64) {
        if (by_score) {
            score_keys<L, P>(a, l, z, top, key, &sum);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                key[i] = z[i] > -INFINITY ? Key64::make((double)z[i], expert_of<L, P>(l, i)) : Key64::kNone;
        }
        if (a.groups > 1) keep_groups<L, P>(a, l, s_keys + (size_t)(threadIdx.x / L) * a.E, key);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) key[i] = Key32::make(z[i], expert_of<L, P>(l, i));
    }

    sort_keys<K, P>(key);
    typename K::type slot[kSlots];
#pragma unroll
    for (int h = 0; h < kSlots; ++h) slot[h] = K::kNone;
    if (P > 8 && a.k <= 8)
        take<K, L, P, (P < 8 ? P : 8)>(a.k, l, key, slot);
    else
        take<K, L, P, (P < kMaxSlots ? P : kMaxSlots)>(a.k, l, key, slot);

    int e[kSlots];
    float zs[kSlots], m = -INFINITY;
#pragma unroll
    for (int h = 0; h < kSlots; ++h) {
        e[h] = -1;
        zs[h] = -INFINITY;
        if (h * L >= a.k) continue;
        const bool taken = slot[h] > K::kNone && on;
        e[h] = taken ? K::index(slot[h]) : -1;
        zs[h] = taken ? tame(raw_logit<BF16>(a.logits, row * a.E + e[h])) : -INFINITY;
        m = fmaxf(m, zs[h]);
    }
    float w[kSlots], all = 0.0f;
    if (a.normalise)
        m = lanes_max<L>(m);
    else
        m = a.sigmoid ? 0.0f : top;
#pragma unroll
    for (int h = 0; h < kSlots; ++h) {
        w[h] = 0.0f;
        if (h * L >= a.k) continue;
        w[h] = e[h] >= 0 ? part(a.sigmoid, zs[h], m) : 0.0f;
        all += w[h];
    }
    if (a.normalise)
        all = lanes_sum<L>(all);
    else
        all = sum;
#pragma unroll
    for (int h = 0; h < kSlots; ++h) {
        const int j = h * L + l;
        if (j < a.k && at < a.T) {
            a.topk_idx[row * a.k + j] = e[h];
            a.weights[row * a.k + j] = e[h] >= 0 ? a.scale * (w[h] / all) : 0.0f;
        }
    }
}

template <int L, int P, bool BF16>
__global__ __launch_bounds__(kRouterThreads) void moedisp_router_backward(RouterArgs a) {
    constexpr int kRows = kRouterThreads / L;
    constexpr int kSlots = (kMaxSlots + L - 1) / L;
    constexpr int V = piece<P>();
    __shared__ __align__(16) float s_d[kRows][L * P];  // the chosen experts' gradients, zeros
    const int l = threadIdx.x % L;
    float* const d_row = s_d[threadIdx.x / L];
    const long long at = (long long)blockIdx.x * kRows + threadIdx.x / L;
    const bool on = at < a.T;
    const size_t row = on ? (size_t)at : 0;
#pragma unroll
    for (int i = 0; i < P; i += 4) *reinterpret_cast<v4f*>(d_row + (i / 4 * L + l) * 4) = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    int e[kSlots];
    float zs[kSlots], g[kSlots], m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int h = 0; h < kSlots; ++h) {
        const int j = h * L + l;
        const bool real = on && j < a.k;
        e[h] = real ? a.topk_idx[row * a.k + j] : -1;
        bad |= e[h] < -1 || e[h] >= a.E;
        if (e[h] >= a.E) e[h] = -1;
        zs[h] = e[h] >= 0 ? tame(raw_logit<BF16>(a.logits, row * a.E + e[h])) : -INFINITY;
        if (!(zs[h] > -INFINITY)) e[h] = -1;  // takes no part
        g[h] = e[h] >= 0 ? a.scale * a.weights[row * a.k + j] : 0.0f;
        m = e[h] >= 0 ? fmaxf(m, zs[h]) : m;
    }
    if (bad) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_EXPERT_ID);

    // softmax of all experts
    const bool whole = !a.sigmoid && !a.normalise;
    float p[P], sum = 1.0f;
    if (whole) {
        load_row<L, P, BF16>(a, row, l, p);
        m = p[0];
#pragma unroll
        for (int i = 1; i < P; ++i) m = fmaxf(m, p[i]);
        m = lanes_max<L>(m);
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            p[i] = exp32(p[i] - m);
            sum += p[i];
        }
        sum = lanes_sum<L>(sum);
    } else if (a.normalise) {
        m = lanes_max<L>(m);
    } else {
        m = 0.0f;
    }
    float s[kSlots], all = 0.0f, mean = 0.0f;
#pragma unroll
    for (int h = 0; h < kSlots; ++h) {
        s[h] = e[h] >= 0 ? part(a.sigmoid, zs[h], m) : 0.0f;
        all += s[h];
    }
    all = a.normalise ? lanes_sum<L>(all) : sum;
    all = all > 0.0f || all != all ? all : 1.0f;
#pragma unroll
    for (int h = 0; h < kSlots; ++h) {
        s[h] /= all;
        mean += g[h] * s[h];
    }
    if (a.normalise || whole) mean = lanes_sum<L>(mean);
    __syncthreads();  // the zeros
#pragma unroll
    for (int h = 0; h < kSlots; ++h) {
        if (e[h] < 0) continue;
        float d = s[h] * (a.normalise ? g[h] - mean : g[h]);
        if (a.sigmoid) d *= part(true, -zs[h], 0.0f);  // 1 - score
        atomicAdd(&d_row[e[h]], d);
    }
    __syncthreads();
    // the wave's other rows may have slots: all lanes of a row agree by now
    const float used = whole && mean != 0.0f ? mean / sum : 0.0f;
    if (!on) return;
#pragma unroll
    for (int c = 0; c < P / V; ++c) {
        const int e0 = (c * L + l) * V;
        if (e0 >= a.E) continue;
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            d[i] = d_row[e0 + i];
            if (used != 0.0f) d[i] -= p[c * V + i] * used;
        }
        if (BF16) {
            uint16_t* o = reinterpret_cast<uint16_t*>(a.d_logits) + row * a.E + e0;
            if (a.vec) {
                if constexpr (V == 8)
                    *reinterpret_cast<v4u*>(o) = v4u{pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]),
                                                     pack_bf16x2(d[4], d[5]), pack_bf16x2(d[6], d[7])};
                else
                    *reinterpret_cast<v2i*>(o) = v2i{(int)pack_bf16x2(d[0], d[1]), (int)pack_bf16x2(d[2], d[3])};
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e0 + i < a.E) o[i] = (uint16_t)pack_bf16x2(d[i], 0.0f);
            }
        } else {
            float* o = reinterpret_cast<float*>(a.d_logits) + row * a.E + e0;
            if (a.vec) {
#pragma unroll
                for (int i = 0; i < V; i += 4) *reinterpret_cast<v4f*>(o + i) = v4f{d[i], d[i + 1], d[i + 2], d[i + 3]};
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e0 + i < a.E) o[i] = d[i];
            }
        }
    }
}

template <int L, int P, bool BF16>
hipError_t launch_shape(RouterArgs a, bool backward, hipStream_t stream) {
    constexpr int kRows = kRouterThreads / L;
    a.vec = a.E % piece<P>() == 0;
    const long long blocks = ((long long)a.T + kRows - 1) / kRows;
    if (!grid_fits(blocks, kRouterThreads)) return hipErrorInvalidConfiguration;
    if (backward) {
        hipLaunchKernelGGL((moedisp_router_backward<L, P, BF16>), dim3((unsigned)blocks), dim3(kRouterThreads), 0,
                           stream, a);
    } else {
        const bool logits_only = a.bias == nullptr && a.groups == 1;
        const size_t lds = a.groups > 1 ? (size_t)kRows * a.E * sizeof(double) : 0;
        a.group_lanes = 1;
        while (2 * a.group_lanes * a.groups <= L) a.group_lanes *= 2;
        if (BF16 && logits_only)
            hipLaunchKernelGGL((moedisp_router<Key32, L, P, true>), dim3((unsigned)blocks), dim3(kRouterThreads), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((moedisp_router<Key64, L, P, BF16>), dim3((unsigned)blocks), dim3(kRouterThreads), lds,
                               stream, a);
    }
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch(const RouterArgs& a, bool backward, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const RouterShape s = router_shape(a.T, a.E);
    if (s.lanes == 16) {
        if (s.per_lane == 4) return launch_shape<16, 4, BF16>(a, backward, stream);
        if (s.per_lane == 8) return launch_shape<16, 8, BF16>(a, backward, stream);
        return launch_shape<16, 16, BF16>(a, backward, stream);
    }
    if (s.per_lane == 4) return launch_shape<64, 4, BF16>(a, backward, stream);
    if (s.per_lane == 8) return launch_shape<64, 8, BF16>(a, backward, stream);
    if (s.per_lane == 16) return launch_shape<64, 16, BF16>(a, backward, stream);
    return launch_shape<64, 64, BF16>(a, backward, stream);
}

}  // namespace

// 16 lanes a row let a wave work on four; a whole wave is quicker where there
// are few rows (256 experts with bias and groups, 1024 rows: 12.5 us a call and
// 6.5; 4096: 12.9 and 10.9; 8192: 16.2 and 18.4.  131072 rows of bf16, both
// directions: 66 and 121).
RouterShape router_shape(int T, int E) {
    if (E <= 64) return {16, 4};
    if (E <= 128) return {16, 8};
    if (E <= 256) return T <= 4096 ? RouterShape{64, 4} : RouterShape{16, 16};
    if (E <= 512) return {64, 8};
    if (E <= 1024) return {64, 16};
    return {64, 64};
}

hipError_t launch_router(const RouterArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch<true>(a, false, stream) : launch<false>(a, false, stream);
}
hipError_t launch_router_backward(const RouterArgs& a, bool bf16, hipStream_t stream) {
    return bf16 ? launch<true>(a, true, stream) : launch<false>(a, true, stream);
}

}  // namespace moedisp
