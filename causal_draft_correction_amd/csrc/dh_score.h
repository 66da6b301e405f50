// Token log-probabilities and entropies of rows: the parts that chunks leave of a row, and what becomes of them.
//
// With y = z / tau, M the row's largest y and one element that has it set apart,
//     So = sum over the other elements of exp(y - M),   T = sum of exp(y - M) (y - M)   (0 for the one set apart)
//     log p_v = y_v - M - log1p(So),   H = log1p(So) - T / (1 + So),   1 - p = So / (1 + So) for the largest
// so that a row that is nearly certain keeps the digits of its small log-probability, entropy and gradient: none of these
// is a difference of numbers near each other.  A chunk takes its largest element out of the sum of all; where less than
// 1/8 is left, it reads the chunk again and takes the sum without it.  (To look for it in the registers first, in every
// chunk, cost 512 bfloat16 rows of 151936 with 20 alternatives 12 us of 49.)
#pragma once

#include "dh_rows.h"

namespace DH_NS {

constexpr double LN2 = 0.69314718055994531, LOG2E = 1.4426950408889634074;

// A chunk: its largest logit m (NaN: the chunk holds a NaN or +inf), s and t as above, t in powers of 2 ((y - M) log2 e);
// (-inf, 0, 0) for a chunk of nothing but -inf.
struct ScorePart {
    float m;
    double s, t;
};

struct Score {
    const int32_t *tokens;
    float *logprob, *entropy;
    float *stats;  // [rows, SCORE_STATS] or NULL
};
constexpr int SCORE_STATS = 8;

__device__ inline bool score_counts(const Rows &rows, const Score &sc, const Place &at)
{
    if (!rows.counts(at.b, at.r))
        return false;
    const int token = sc.tokens[at.row];
    return token >= 0 && token < rows.V;
}

// The thread's exponentials and exponentials times exponents.  (An exponent of -inf gives 0: the product takes one that
// is finite.)
template <typename T, bool SMALL, int NV>
__device__ inline void sum_scores(typename Vec<T>::raw (&x)[NV], const Expo &ex, const Scale &sc, float &s, float &t)
{
    forget(x);
    s = t = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float one = 0.f, two = 0.f;
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) {
            const float y = ex.exponent<SMALL>(Vec<T>::get(x[u], e), sc), p = __builtin_amdgcn_exp2f(y);
            one = e ? one + p : p;
            two = e ? fmaf(p, fmaxf(y, -1000.f), two) : p * fmaxf(y, -1000.f);
        }
        s += one;
        t += two;
    }
}

// The same over the thread's elements of chunk c, read again one by one, without one equal to m, the block's largest: the
// first such of the first wave that has one (`red_m`: the waves' largest), of its first lane (`mine`: the thread's).
template <typename T, int NTB>
__device__ inline void sums_without(const T *row, int V, int c, int cvec, float mine, float m, const float *red_m,
                                    const Expo &ex, const Scale &sc, float &s, float &t)
{
    int first = NTB / 64 - 1;
#pragma unroll
    for (int w = NTB / 64 - 2; w >= 0; --w)
        first = red_m[w] == m ? w : first;
    const uint64_t has = __ballot(mine == m);
    bool skip = static_cast<int>(threadIdx.x >> 6) == first &&
                static_cast<int>(threadIdx.x & 63) == __ffsll(static_cast<unsigned long long>(has)) - 1;
    s = t = 0.f;
    // two vectors at a time: more would take registers, and waves, from the common way
    constexpr int STEP = 2;
    const int64_t v0 = static_cast<int64_t>(c) * cvec * Vec<T>::N, left = V - v0;
    const int n = left < static_cast<int64_t>(cvec) * Vec<T>::N ? static_cast<int>(left) : cvec * Vec<T>::N;
#pragma unroll 1
    for (int i = 0; i * STEP * NTB * Vec<T>::N < n; ++i) {
        typename Vec<T>::raw x[STEP];
        load_chunk<T, STEP, NTB, true>(x, row + v0, n, i, STEP * NTB);
#pragma unroll
        for (int u = 0; u < STEP; ++u) {
            float one = 0.f, two = 0.f;
#pragma unroll
            for (int e = 0; e < Vec<T>::N; ++e) {
                float z = Vec<T>::get(x[u], e);
                const bool it = skip && z == m;
                skip = skip && !it;
                z = it ? NEG_INF : z;
                const float y = ex.small ? ex.exponent<true>(z, sc) : ex.exponent<false>(z, sc);
                const float p = __builtin_amdgcn_exp2f(y);
                one += p;
                two = fmaf(p, fmaxf(y, -1000.f), two);
            }
            s += one;
            t += two;
        }
    }
}

// A block's part, of chunk c of a row: its threads' elements x, each thread's largest one (`mine`) and the block's (m),
// `red_m` the waves'.  odd: a NaN, or +inf more than once.
template <typename T, int NV, int NTB>
__device__ inline ScorePart block_score(typename Vec<T>::raw (&x)[NV], const T *row, int V, int c, int cvec, float mine,
                                        float m, const float *red_m, double (*red)[2], const Expo &ex, const Scale &sc,
                                        bool &odd)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    double s, t;
    const auto over_block = [&](float s1, float t1) {
        s = wave_sum_f64(s1), t = wave_sum_f64(t1);
        if (lane == 0)
            red[wave][0] = s, red[wave][1] = t;
        __syncthreads();
        s = t = 0.0;
#pragma unroll
        for (int w = 0; w < NTB / 64; ++w)
            s += red[w][0], t += red[w][1];
    };
    float s1, t1;
    if (ex.small)
        sum_scores<T, true>(x, ex, sc, s1, t1);
    else
        sum_scores<T, false>(x, ex, sc, s1, t1);
    over_block(s1, t1);
    odd = s != s;
    if (odd || m == -NEG_INF)
        return ScorePart{__builtin_nanf(""), 0.0, 0.0};
    if (m == NEG_INF)
        return ScorePart{NEG_INF, 0.0, 0.0};
    const float y = ex.small ? ex.exponent<true>(m, sc) : ex.exponent<false>(m, sc), p = __builtin_amdgcn_exp2f(y);
    s -= p, t -= static_cast<double>(p) * y;
    if (s < 0.125) {
        sums_without<T, NTB>(row, V, c, cvec, mine, m, red_m, ex, sc, s1, t1);
        __syncthreads();
        over_block(s1, t1);
    }
    // (the exponents have Expo's c in them)
    return ScorePart{m, s * ex.fix(sc), (t - ex.off(sc) * s) * ex.fix(sc)};
}

__device__ inline ScorePart first_part(const ScorePart *parts, int nch)
{
    const int lane = threadIdx.x & 63;
    return lane < nch ? parts[lane] : ScorePart{NEG_INF, 0.0, 0.0};
}

// A row's part from its chunks', in 64 bits; every lane of the wave gets it.
__device__ inline ScorePart join_parts(const ScorePart &first, const ScorePart *parts, int nch, double inv_tau)
{
    const int lane = threadIdx.x & 63;
    float mx = fmaxf(NEG_INF, first.m);
    bool bad = first.m != first.m;
    for (int c = lane + 64; c < nch; c += 64) {
        const float v = parts[c].m;
        bad |= v != v;
        mx = fmaxf(mx, v);
    }
    const float m = wave_max(mx);
    if (__ballot(bad))
        return ScorePart{__builtin_nanf(""), 0.0, 0.0};
    double s = 0.0, t = 0.0;
    int at_top = 0;
    auto add = [&](const ScorePart &p) {
        if (p.m > NEG_INF) {
            const double y = (static_cast<double>(p.m) - m) * inv_tau, w = p.m == m ? 1.0 : exp(y);
            // the element set apart of a chunk below the top, or of a second one at it, is one of the others
            at_top += p.m == m;
            s += w * p.s + (p.m == m ? 0.0 : w);
            t += w * p.t + (p.m == m ? 0.0 : w * (p.s + 1.0) * y * LOG2E);
        }
    };
    add(first);
    for (int c = lane + 64; c < nch; c += 64)
        add(parts[c]);
    const double tops = wave_sum_f64(static_cast<double>(at_top));
    s = wave_sum_f64(s) + (tops > 1.0 ? tops - 1.0 : 0.0);
    return ScorePart{m, s, wave_sum_f64(t)};
}

// log p of a logit of the row (NaN in rows without a distribution, -inf in rows of nothing but -inf).
__device__ inline double log_prob(float z, const ScorePart &row, double log_s, double inv_tau)
{
    if (row.m != row.m)
        return __builtin_nan("");
    if (z == NEG_INF)
        return -__builtin_huge_val();
    return (static_cast<double>(z) - row.m) * inv_tau - log_s;
}

__device__ inline void no_score(const Score &sc, int row)
{
    sc.logprob[row] = sc.entropy[row] = 0.f;
    if (sc.stats) {
        const float4 zero = {0.f, 0.f, 0.f, 0.f};
        float4 *st = reinterpret_cast<float4 *>(sc.stats + static_cast<int64_t>(row) * SCORE_STATS);
        st[0] = st[1] = zero;
    }
}

// What the backward pass needs of a row:
//     { M (as a logit), 1 / S, H - log S, 1 (0: no gradient), p, 1 - p, p (log p + H) of the token, 0 }
__device__ inline void score_stats(const ScorePart &row, double log_s, double entropy, double logprob, bool top,
                                   float (&st)[SCORE_STATS])
{
    const double p = exp(logprob), S = 1.0 + row.s;
    const bool none = row.m == NEG_INF;
    st[0] = none ? 0.f : row.m;
    st[1] = static_cast<float>(row.m != row.m ? __builtin_nan("") : 1.0 / S);
    st[2] = static_cast<float>(entropy - log_s);
    st[3] = none ? 0.f : 1.f;
    st[4] = static_cast<float>(p);
    st[5] = static_cast<float>(top ? row.s / S : 1.0 - p);
    st[6] = static_cast<float>(p == 0.0 ? 0.0 : p * (logprob + entropy));
    st[7] = 0.f;
}

// Results of a row from its part, by one thread.
__device__ inline void put_score(const Score &sc, int at, float z_token, const ScorePart &row, double log_s,
                                 double inv_tau, float *stats)
{
    const bool none = row.m == NEG_INF;
    const double logprob = none ? -__builtin_huge_val() : log_prob(z_token, row, log_s, inv_tau);
    const double entropy = row.m != row.m ? __builtin_nan("") : none ? 0.0 : log_s - LN2 * row.t / (1.0 + row.s);
    sc.logprob[at] = static_cast<float>(logprob);
    sc.entropy[at] = static_cast<float>(entropy);
    if (stats) {
        float st[SCORE_STATS];
        score_stats(row, log_s, entropy, logprob, z_token == row.m, st);
#pragma unroll
        for (int i = 0; i < SCORE_STATS; ++i)
            stats[i] = st[i];
    }
}

}  // namespace DH_NS
