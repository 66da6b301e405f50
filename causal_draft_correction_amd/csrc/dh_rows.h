// Rows of logits in chunks: what the kernels over vocabulary rows share.
//
// A row of V logits (float32 or bfloat16, contiguous, at any element address) is split into `nch` chunks of
// `cvec` 16-byte vectors, one 256-thread block each; a thread keeps its NV vectors of the chunk in registers
// (vector u * 256 + thread of the chunk), so that the maximum, the sum of exponentials and the selection are
// taken from one reading of the row.
#pragma once

#include "dh_common.h"

#include <cmath>

namespace DH_NS {

constexpr float NEG_INF = -__builtin_huge_valf();

// [B, R, V] logits: element strides of a batch entry and of a row; n_rows: rows of each batch entry that
// count (NULL = all R).
struct Rows {
    const void *data;
    int64_t bs, rs;
    int R, V;
    const int32_t *n_rows;
    __device__ bool counts(int b, int r) const { return !n_rows || r < n_rows[b]; }
};

// How a row is split: nch chunks of cvec vectors (the last one may hold fewer).
struct Split {
    int nch, cvec, nv;
};

// A vector of 16 bytes at any element address: the compiler's unaligned global loads and stores.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    typedef float raw __attribute__((ext_vector_type(4)));
    typedef float mem __attribute__((ext_vector_type(4), aligned(4)));
    __device__ static raw fill() { return raw{NEG_INF, NEG_INF, NEG_INF, NEG_INF}; }
    __device__ static float get(const raw &x, int e) { return x[e]; }
    __device__ static void set(raw &x, int e, float f) { x[e] = f; }
    __device__ static float one(const float *p) { return *p; }
    __device__ static void put(float *p, float f) { *p = f; }
};
template <>
struct Vec<bf16s> {
    static constexpr int N = 8;
    typedef uint32_t raw __attribute__((ext_vector_type(4)));
    typedef uint32_t mem __attribute__((ext_vector_type(4), aligned(2)));
    __device__ static raw fill() { return raw{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u}; }
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
    __device__ static float one(const bf16s *p) { return __uint_as_float(static_cast<uint32_t>(p->bits) << 16); }
    __device__ static void put(bf16s *p, float f) { p->bits = static_cast<uint16_t>(bits(f)); }
};

template <typename T>
__device__ inline const T *row_at(const Rows &rows, int b, int r)
{
    return static_cast<const T *>(rows.data) + b * rows.bs + r * rows.rs;
}

// The thread's vectors of chunk c; places past the chunk or the row hold -inf.
template <typename T, int NV>
__device__ inline void load_chunk(typename Vec<T>::raw (&x)[NV], const T *row, int V, int c, int cvec)
{
    typedef Vec<T> VT;
    const int first = c * cvec;                                // the chunk's first vector
    const int full = V / VT::N;                                // whole vectors of the row
    const int n = full - first < cvec ? full - first : cvec;   // whole vectors of this chunk
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int i = u * NT + static_cast<int>(threadIdx.x);
        x[u] = VT::fill();
        if (i < n)
            x[u] = __builtin_nontemporal_load(
                reinterpret_cast<const typename VT::mem *>(row + static_cast<int64_t>(first + i) * VT::N));
    }
    const int tail = V - full * VT::N;
    if (tail && n >= 0 && n < cvec) {  // the row's last elements, element by element
        typename VT::raw t = VT::fill();
        if (n % NT == static_cast<int>(threadIdx.x)) {
#pragma unroll
            for (int e = 0; e < VT::N; ++e)
                if (e < tail)
                    VT::set(t, e, VT::one(row + static_cast<int64_t>(full) * VT::N + e));
#pragma unroll
            for (int u = 0; u < NV; ++u)
                if (u * NT + static_cast<int>(threadIdx.x) == n)
                    x[u] = t;
        }
    }
}

// First element of chunk c and the element after its last.
template <typename T>
__device__ inline int chunk_begin(int c, int cvec, int V)
{
    const int64_t v = static_cast<int64_t>(c) * cvec * Vec<T>::N;
    return v < V ? static_cast<int>(v) : V;
}

// exp(d / tau) as 2^(d log2(e) / tau), d <= 0; the factor in two parts, since its own rounding would be an error
// common to all terms of a sum.  Both parts are above 0, so that d = -inf gives 0.  (v_exp_f32 flushes results
// below 2^-126.)
struct Scale {
    float hi, lo;
};
inline Scale scale_of(float tau)
{
    const double s = 1.4426950408889634074 / static_cast<double>(tau);
    Scale sc;
    sc.hi = static_cast<float>(s);
    if (static_cast<double>(sc.hi) >= s)
        sc.hi = std::nextafterf(sc.hi, 0.f);
    sc.lo = static_cast<float>(s - static_cast<double>(sc.hi));
    return sc;
}
__device__ inline float exp_scaled(float d, const Scale &s)
{
    return __builtin_amdgcn_exp2f(fmaf(d, s.hi, d * s.lo));
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

__device__ inline double wave_sum_f64(double v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}

// What the chunks of a row leave of its log-sum-exp: the maximum m (NaN: the chunk holds a NaN) and
// s = sum exp((z - m) / tau), (-inf, 0) for a chunk of nothing but -inf.
struct Part {
    float m, s;
};

// A row's maximum and its sum of exponentials from its chunks' parts, in 64 bits; every lane of the wave gets
// them.  A NaN part makes both NaN.
__device__ inline void join_parts(const Part *parts, int nch, double inv_tau, float &m, double &s)
{
    const int lane = threadIdx.x & 63;
    float mx = NEG_INF;
    bool bad = false;
    for (int c = lane; c < nch; c += 64) {
        const float v = parts[c].m;
        bad |= v != v;
        mx = fmaxf(mx, v);
    }
    m = wave_max(mx);
    bad = __ballot(bad) != 0;
    double t = 0.0;
    for (int c = lane; c < nch; c += 64) {
        const Part p = parts[c];
        if (p.m > NEG_INF)
            t += static_cast<double>(p.s) * (p.m == m ? 1.0 : exp((static_cast<double>(p.m) - m) * inv_tau));
    }
    s = wave_sum_f64(t);
    if (bad)
        s = __builtin_nan(""), m = __builtin_nanf("");
}

}  // namespace DH_NS
