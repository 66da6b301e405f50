// Rows of logits in chunks: what the kernels over vocabulary rows share.
//
// A row of V logits (float32 or bfloat16, contiguous, at any element address) is split into `nch` chunks of
// `cvec` 16-byte vectors, one 256-thread block each; a thread keeps its NV vectors of the chunk in registers
// (vector u * 256 + thread of the chunk), so that the maximum, the sum of exponentials and the selection are
// taken from one reading of the row.  The vectors are loaded at the row's own alignment: 1024 bf16 rows of 50021
// at odd addresses take 32.0 us for their sums, at 16-byte addresses 30.8 us, which pays for no second path.
#pragma once

#include "dh_common.h"

#include <cmath>

#include "../../include/domino_head.h"

namespace DH_NS {

constexpr float NEG_INF = -__builtin_huge_valf();

// Division of block numbers (below 2^31) by a divisor known on the host: with 2^shift the power of two not below
// it and mul = floor(2^32 (2^shift - divisor) / divisor) + 1, n / divisor = (mulhi(n, mul) + n) >> shift.
struct Divisor {
    uint32_t d, mul, shift;
    __device__ uint32_t quotient(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};
inline Divisor divisor(uint32_t d)
{
    Divisor v;
    v.d = d;
    v.shift = 0;
    while ((uint64_t(1) << v.shift) < d)
        ++v.shift;
    v.mul = static_cast<uint32_t>((uint64_t(1) << 32) * ((uint64_t(1) << v.shift) - d) / d + 1);
    return v;
}

// A row: row b R + r of the launch's.
struct Place {
    int b, r, row;
};

// [B, R, V] logits: element strides of a batch entry and of a row; n_rows: rows of each batch entry that
// count (NULL = all R).
struct Rows {
    const void *data;
    int64_t bs, rs;
    int R, V;
    const int32_t *n_rows;
    bool across;    // the order of a launch's rows: through the batch entries first
    Divisor by;     // B, or R
    __device__ bool counts(int b, int r) const { return !n_rows || r < n_rows[b]; }
    // The i-th row of a launch.  Where some rows may be left out, these are the later ones of a batch entry: with the
    // batch entries first, the blocks with work come first and spread evenly over the device (24 x 16 bf16 rows of
    // 50021, half of them left out: 17.3 us by batch entries, 14.4 us across them).
    __device__ Place place(uint32_t i) const
    {
        const int q = static_cast<int>(by.quotient(i)), rem = static_cast<int>(i - q * by.d);
        const int b = across ? rem : q, r = across ? q : rem;
        return Place{b, r, b * R + r};
    }
};
inline Rows rows_of(const domino_logits &lg, const int32_t *n_rows, bool across)
{
    Rows r;
    r.data = lg.data;
    r.bs = lg.batch_stride;
    r.rs = lg.row_stride;
    r.R = lg.R;
    r.V = lg.V;
    r.n_rows = n_rows;
    r.across = across;
    r.by = divisor(static_cast<uint32_t>(across ? lg.B : lg.R));
    return r;
}

// How a row is split: nch chunks of cvec vectors (the last one may hold fewer), nv of them a thread; one block each,
// the chunks of a row one after the other.
struct Split {
    int nch, cvec, nv;
    Divisor by;
};
inline Split split(int64_t nvec, int64_t n)
{
    Split sp;
    sp.cvec = static_cast<int>((nvec + n - 1) / n);
    sp.nch = static_cast<int>((nvec + sp.cvec - 1) / sp.cvec);
    sp.nv = (sp.cvec + NT - 1) / NT;
    sp.by = divisor(static_cast<uint32_t>(sp.nch));
    return sp;
}

// A vector of 16 bytes at any element address: the compiler's unaligned global loads and stores.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    typedef float raw __attribute__((ext_vector_type(4)));
    typedef float mem __attribute__((ext_vector_type(4), aligned(4)));
    __device__ static raw fill() { return raw{NEG_INF, NEG_INF, NEG_INF, NEG_INF}; }
    // element i of vectors stored as words
    __device__ static float word_at(const uint32_t *words, int i) { return __uint_as_float(words[i]); }
    // the largest element and `m` (NaN are passed over)
    __device__ static float max_with(const raw &x, float m)
    {
        return fmaxf(fmaxf(fmaxf(fmaxf(m, x[0]), x[1]), x[2]), x[3]);
    }
    __device__ static float get(const raw &x, int e) { return x[e]; }
    __device__ static void set(raw &x, int e, float f) { x[e] = f; }
    template <typename F>
    __device__ static void map(raw &x, F f)
    {
#pragma unroll
        for (int e = 0; e < N; ++e)
            x[e] = f(x[e]);
    }
    __device__ static float one(const float *p) { return *p; }
    __device__ static void put(float *p, float f) { *p = f; }
};
template <>
struct Vec<bf16s> {
    static constexpr int N = 8;
    typedef uint32_t raw __attribute__((ext_vector_type(4)));
    typedef uint32_t mem __attribute__((ext_vector_type(4), aligned(2)));
    __device__ static raw fill() { return raw{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u}; }
    __device__ static float word_at(const uint32_t *words, int i)
    {
        return __uint_as_float((i & 1) ? (words[i >> 1] & 0xFFFF0000u) : (words[i >> 1] << 16));
    }
    __device__ static float get(const raw &x, int e)
    {
        return __uint_as_float((e & 1) ? (x[e >> 1] & 0xFFFF0000u) : (x[e >> 1] << 16));
    }
    // rounds to nearest even (the hardware conversion; a NaN stays one)
    __device__ static uint32_t bits(float f)
    {
        return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f)));
    }
    __device__ static void set(raw &x, int e, float f)
    {
        x[e >> 1] = (e & 1) ? ((x[e >> 1] & 0xFFFFu) | (bits(f) << 16)) : ((x[e >> 1] & 0xFFFF0000u) | bits(f));
    }
    // the largest element and `m` (NaN are passed over)
    __device__ static float max_with(const raw &x, float m)
    {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            m = fmaxf(fmaxf(m, get(x, i)), get(x, i + 1));
        return m;
    }
    template <typename F>
    __device__ static void map(raw &x, F f)
    {
        typedef __bf16 pair __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const pair p = {static_cast<__bf16>(f(get(x, 2 * i))), static_cast<__bf16>(f(get(x, 2 * i + 1)))};
            x[i] = __builtin_bit_cast(uint32_t, p);
        }
    }
    __device__ static float one(const bf16s *p) { return __uint_as_float(static_cast<uint32_t>(p->bits) << 16); }
    __device__ static void put(bf16s *p, float f) { p->bits = static_cast<uint16_t>(bits(f)); }
};

template <typename T>
__device__ inline const T *row_at(const Rows &rows, const Place &at)
{
    return static_cast<const T *>(rows.data) + at.b * rows.bs + at.r * rows.rs;
}

// The thread's vectors of chunk c (vectors c * cvec on) for blocks of NTB threads; places past the chunk or the
// row hold -inf.  KEEP: the row is read again soon, so it may stay in the caches.
template <typename T, int NV, int NTB = NT, bool KEEP = false>
__device__ inline void load_chunk(typename Vec<T>::raw (&x)[NV], const T *row, int V, int c, int cvec)
{
    typedef Vec<T> VT;
    const int first = c * cvec;                                // the chunk's first vector
    const int full = V / VT::N;                                // whole vectors of the row
    const int n = full - first < cvec ? full - first : cvec;   // whole vectors of this chunk
    const T *start = row + static_cast<int64_t>(first) * VT::N;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int i = u * NTB + static_cast<int>(threadIdx.x);
        // (the chunk's start is the same in every thread, the rest 32 bits)
        const auto *p = reinterpret_cast<const typename VT::mem *>(start + static_cast<uint32_t>(i) * VT::N);
        x[u] = VT::fill();
        if (i < n)
            x[u] = KEEP ? *p : __builtin_nontemporal_load(p);
    }
    const int tail = V - full * VT::N;
    if (tail && n >= 0 && n < cvec) {  // the row's last elements, element by element
        typename VT::raw t = VT::fill();
        if (n % NTB == static_cast<int>(threadIdx.x)) {
#pragma unroll
            for (int e = 0; e < VT::N; ++e)
                if (e < tail)
                    VT::set(t, e, VT::one(row + static_cast<int64_t>(full) * VT::N + e));
#pragma unroll
            for (int u = 0; u < NV; ++u)
                if (u * NTB + static_cast<int>(threadIdx.x) == n)
                    x[u] = t;
        }
    }
}

// Stores the thread's vectors of chunk c = elements [v0, v1).
template <typename T, int NV, int NTB = NT>
__device__ inline void store_chunk(const typename Vec<T>::raw (&x)[NV], T *row, int v0, int v1)
{
    typedef Vec<T> VT;
    T *start = row + v0;
    const int n = v1 - v0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int i = (u * NTB + static_cast<int>(threadIdx.x)) * VT::N;
        if (i + VT::N <= n) {
            __builtin_nontemporal_store(x[u], reinterpret_cast<typename VT::mem *>(start + static_cast<uint32_t>(i)));
        } else if (i < n) {
#pragma unroll
            for (int e = 0; e < VT::N; ++e)
                if (i + e < n)
                    VT::put(start + i + e, VT::get(x[u], e));
        }
    }
}

// Makes the vectors' values opaque, so that bfloat16 elements are widened again where they are next used, and not
// kept in registers as floats.
template <typename V, int NV>
__device__ inline void forget(V (&x)[NV])
{
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            auto w = x[u][i];
            asm("" : "+v"(w));
            x[u][i] = w;
        }
}

// First element of chunk c and the element after its last.
template <typename T>
__device__ inline int chunk_begin(int c, int cvec, int V)
{
    const int64_t v = static_cast<int64_t>(c) * cvec * Vec<T>::N;
    return v < V ? static_cast<int>(v) : V;
}

// exp((z - ref) / tau) as a power of 2, with s = log2(e) / tau.
//
// Where |ref s| < 1024 (SMALL) it is 2^(z near + c): near is s rounded to float32, c = -ref near rounded, so that an
// element takes one fused multiply-add.  The rounding of c is the same factor in every term of a sum, and taken
// out of it (fix); that of near weighs up to |ln q| 2^-24 in a term q, below 6e-7 of a sum over any distribution of
// 2^19 elements (n terms exp(-d) beside a term 1 weigh at most d - 1 where n exp(-d) = d - 1, which is 9.8); at
// tau = 1, where near is off by 2^-26.2 of itself, 1.3e-7.
// Elsewhere it is 2^(d hi + d lo) with d = z - ref, hi + lo = s and both above 0, so that d = -inf gives 0.
// (v_exp_f32 flushes results below 2^-126.)
struct Scale {
    float near, hi, lo;
};
inline Scale scale_of(double tau)
{
    const double s = 1.4426950408889634074 / tau;
    Scale sc;
    sc.near = sc.hi = static_cast<float>(s);
    if (static_cast<double>(sc.hi) >= s)
        sc.hi = std::nextafterf(sc.hi, 0.f);
    sc.lo = static_cast<float>(s - static_cast<double>(sc.hi));
    return sc;
}
struct Expo {
    float ref, c;
    bool small;
    __device__ Expo(float r, const Scale &s) : ref(r), c(-r * s.near), small(fabsf(r * s.near) < 1024.f) {}
    // the power of 2
    template <bool SMALL>
    __device__ float exponent(float z, const Scale &s) const
    {
        if constexpr (SMALL)
            return fmaf(z, s.near, c);
        const float d = z - ref;
        return fmaf(d, s.hi, d * s.lo);
    }
    template <bool SMALL>
    __device__ float at(float z, const Scale &s) const
    {
        return __builtin_amdgcn_exp2f(exponent<SMALL>(z, s));
    }
    // by how much exponent() is too large everywhere
    __device__ double off(const Scale &s) const
    {
        return small ? static_cast<double>(c) + static_cast<double>(ref) * s.near : 0.0;
    }
    // what a sum of at() has to be multiplied by
    __device__ double fix(const Scale &s) const
    {
        const double y = 0.69314718055994531 * (static_cast<double>(c) + static_cast<double>(ref) * s.near);
        return small ? 1.0 - y + 0.5 * y * y : 1.0;
    }
};

// Sum of the thread's exponentials, vector by vector.
template <typename T, bool SMALL, int NV>
__device__ inline float sum_exps(typename Vec<T>::raw (&x)[NV], const Expo &ex, const Scale &sc)
{
    forget(x);
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float one = ex.at<SMALL>(Vec<T>::get(x[u], 0), sc);
#pragma unroll
        for (int e = 1; e < Vec<T>::N; ++e)
            one += ex.at<SMALL>(Vec<T>::get(x[u], e), sc);
        s += one;
    }
    return s;
}

__device__ inline float wave_max(float v)
{
    v = fmaxf(v, dpp_f32<DPP_QUAD_XOR1>(v));
    v = fmaxf(v, dpp_f32<DPP_QUAD_XOR2>(v));
    v = fmaxf(v, dpp_f32<DPP_HALF_MIRROR>(v));
    v = fmaxf(v, dpp_f32<DPP_ROW_MIRROR>(v));
    uint32_t a, b;
    row_pair_values(__float_as_uint(v), a, b);
    v = fmaxf(__uint_as_float(a), __uint_as_float(b));
    half_values(__float_as_uint(v), a, b);
    return fmaxf(__uint_as_float(a), __uint_as_float(b));
}

template <int CTRL>
__device__ inline double dpp_f64(double v)
{
    return __builtin_bit_cast(double, dpp_u64<CTRL>(__builtin_bit_cast(uint64_t, v)));
}
// The values of the even and odd row of a row pair, and of the lower and upper half of the wave.
__device__ inline void row_pair_values(double v, double &even, double &odd)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t el, ol, eh, oh;
    row_pair_values(static_cast<uint32_t>(u), el, ol);
    row_pair_values(static_cast<uint32_t>(u >> 32), eh, oh);
    even = __builtin_bit_cast(double, (static_cast<uint64_t>(eh) << 32) | el);
    odd = __builtin_bit_cast(double, (static_cast<uint64_t>(oh) << 32) | ol);
}
__device__ inline void half_values(double v, double &lo, double &hi)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t ll, hl, lh, hh;
    half_values(static_cast<uint32_t>(u), ll, hl);
    half_values(static_cast<uint32_t>(u >> 32), lh, hh);
    lo = __builtin_bit_cast(double, (static_cast<uint64_t>(lh) << 32) | ll);
    hi = __builtin_bit_cast(double, (static_cast<uint64_t>(hh) << 32) | hl);
}

// Sum over the wave, the same bits in every lane.
__device__ inline double wave_sum_f64(double v)
{
    v += dpp_f64<DPP_QUAD_XOR1>(v);
    v += dpp_f64<DPP_QUAD_XOR2>(v);
    v += dpp_f64<DPP_HALF_MIRROR>(v);
    v += dpp_f64<DPP_ROW_MIRROR>(v);
    double a, b;
    row_pair_values(v, a, b);
    half_values(a + b, a, b);
    return a + b;
}

// Maximum over the wave; NaN operands are passed over.
__device__ inline double wave_max_f64(double v)
{
    v = fmax(v, dpp_f64<DPP_QUAD_XOR1>(v));
    v = fmax(v, dpp_f64<DPP_QUAD_XOR2>(v));
    v = fmax(v, dpp_f64<DPP_HALF_MIRROR>(v));
    v = fmax(v, dpp_f64<DPP_ROW_MIRROR>(v));
    double a, b;
    row_pair_values(v, a, b);
    half_values(fmax(a, b), a, b);
    return fmax(a, b);
}

// What the chunks of a row leave of its log-sum-exp: the maximum m (NaN: the chunk holds a NaN) and
// s = sum exp((z - m) / tau), (-inf, 0) for a chunk of nothing but -inf.
struct Part {
    float m;
    double s;
};

// The first part a lane has to join (loaded early, ahead of what else the caller waits for).
__device__ inline Part first_part(const Part *parts, int nch)
{
    const int lane = threadIdx.x & 63;
    return lane < nch ? parts[lane] : Part{NEG_INF, 0.0};
}

// A row's maximum and its sum of exponentials from its chunks' parts, in 64 bits; every lane of the wave gets
// them.  A NaN part makes both NaN.
__device__ inline void join_parts(const Part &first, const Part *parts, int nch, double inv_tau, float &m, double &s)
{
    const int lane = threadIdx.x & 63;
    float mx = fmaxf(NEG_INF, first.m);
    bool bad = first.m != first.m;
    for (int c = lane + 64; c < nch; c += 64) {
        const float v = parts[c].m;
        bad |= v != v;
        mx = fmaxf(mx, v);
    }
    m = wave_max(mx);
    bad = __ballot(bad) != 0;
    double t = 0.0;
    if (first.m > NEG_INF)
        t = first.s * (first.m == m ? 1.0 : exp((static_cast<double>(first.m) - m) * inv_tau));
    for (int c = lane + 64; c < nch; c += 64) {
        const Part p = parts[c];
        if (p.m > NEG_INF)
            t += p.s * (p.m == m ? 1.0 : exp((static_cast<double>(p.m) - m) * inv_tau));
    }
    s = wave_sum_f64(t);
    if (bad)
        s = __builtin_nan(""), m = __builtin_nanf("");
}

}  // namespace DH_NS
