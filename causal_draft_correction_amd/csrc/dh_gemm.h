// Products of rows on the matrix cores, with an epilogue: D[j][i] = sum_k A(i, k) B(j, k), the kernels of domino_linear.
//
// An operand lies along k (its row i holds k = 0, 1, ...: x and w of a forward pass) or across k (its row k holds
// i = 0, 1, ...: w where the sum goes over its rows, both where it goes over the batch).  A block takes a tile of
// BI x BJ and BK of k at a time: global memory -> registers (the next step's while this one is multiplied) -> LDS as
// bfloat16, transposed where the operand lies across k, -> v_mfma_f32_16x16x32_bf16, summed in float32.
//
// float32 operands are cut into three bfloat16 planes, x = h + m + l, each the rounded remainder of those before: that
// is all of x's 24 bits, and every product of two planes is exact in float32.  A float32 and a bfloat16 operand take 3
// products, two float32 operands the 6 that weigh at least 2^-18 of the first (the three left out weigh at most 2^-26 of
// it): 0.8 and 0.4 PFLOP/s at the bfloat16 rate, where the float32 instruction reaches 0.16.
#pragma once

#include "dh_linear.h"
#include "dh_rows.h"

namespace DH_NS {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Rows at data + b bs + r rs, row b R + r; flat: all rs apart.
struct Mat {
    const void *data;
    int64_t bs, rs;
    Divisor by;  // R
    bool flat, f32;
    __device__ int64_t row(int i) const
    {
        if (flat)
            return i * rs;
        const int b = static_cast<int>(by.quotient(static_cast<uint32_t>(i)));
        return b * bs + (i - b * static_cast<int>(by.d)) * rs;
    }
};
inline Mat mat_of(const domino_rows &m)
{
    Mat t;
    t.data = m.data;
    t.bs = m.batch_stride;
    t.rs = m.R == 1 ? m.batch_stride : m.row_stride;
    t.by = divisor(static_cast<uint32_t>(m.R));
    t.flat = m.R == 1 || m.B <= 1 || m.batch_stride == m.R * m.row_stride;
    t.f32 = m.dtype == DOMINO_F32;
    return t;
}

// ---- epilogue ----

__device__ inline float act_of(float a, int act)
{
    if (act == DOMINO_SILU)
        return a / (1.f + expf(-a));
    if (act == DOMINO_GELU)
        return 0.5f * a * erfcf(-0.70710678f * a);
    return act == DOMINO_RELU ? (a > 0.f || a != a ? a : 0.f) : a;
}
__device__ inline float slope_of(float a, int act)
{
    if (act == DOMINO_SILU) {
        const float s = 1.f / (1.f + expf(-a));
        // (1 - s as a sigmoid of its own: far from 0 it keeps its digits)
        return s * (1.f + a * (1.f / (1.f + expf(a))));
    }
    if (act == DOMINO_GELU)
        return 0.5f * erfcf(-0.70710678f * a) + a * 0.39894228f * expf(-0.5f * a * a);
    return act == DOMINO_RELU ? (a > 0.f ? 1.f : a != a ? a : 0.f) : 1.f;
}

// n (at most 4) elements from o of a row.
__device__ inline void get4(const void *data, bool f32, int64_t o, int n, float (&f)[4])
{
    if (f32) {
        const float *p = static_cast<const float *>(data) + o;
        if (n >= 4) {
            const Vec<float>::raw x = *reinterpret_cast<const Vec<float>::mem *>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = x[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = e < n ? p[e] : 0.f;
        }
    } else {
        typedef uint32_t two __attribute__((ext_vector_type(2), aligned(2)));
        const bf16s *p = static_cast<const bf16s *>(data) + o;
        if (n >= 4) {
            const two x = *reinterpret_cast<const two *>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = __uint_as_float(e & 1 ? x[e >> 1] & 0xFFFF0000u : x[e >> 1] << 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = e < n ? Vec<bf16s>::one(p + e) : 0.f;
        }
    }
}
__device__ inline void put4(const void *data, bool f32, int64_t o, int n, const float (&f)[4])
{
    if (f32) {
        float *p = static_cast<float *>(const_cast<void *>(data)) + o;
        if (n >= 4) {
            *reinterpret_cast<Vec<float>::mem *>(p) = Vec<float>::raw{f[0], f[1], f[2], f[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n)
                    p[e] = f[e];
        }
    } else {
        typedef uint32_t two __attribute__((ext_vector_type(2), aligned(2)));
        bf16s *p = static_cast<bf16s *>(const_cast<void *>(data)) + o;
        if (n >= 4) {
            *reinterpret_cast<two *>(p) = two{Vec<bf16s>::bits(f[0]) | (Vec<bf16s>::bits(f[1]) << 16),
                                              Vec<bf16s>::bits(f[2]) | (Vec<bf16s>::bits(f[3]) << 16)};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n)
                    Vec<bf16s>::put(p + e, f[e]);
        }
    }
}

// What becomes of the sums: pre = sum + bias, D = act(pre) + residual.
struct Epilogue {
    Mat out, pre, residual;  // data NULL: none
    const void *bias;
    bool bias_f32;
    int act;
};

// Elements i .. i + 3 (those below I) of row j.
__device__ inline void emit(const Epilogue &e, int i, int I, int64_t o_out, int64_t o_pre, int64_t o_res, float (&v)[4])
{
    const int n = I - i;
    float f[4];
    if (e.bias) {
        get4(e.bias, e.bias_f32, i, n, f);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] += f[u];
    }
    if (e.pre.data)
        put4(e.pre.data, e.pre.f32, o_pre + i, n, v);
    if (e.act != DOMINO_NO_ACT)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = act_of(v[u], e.act);
    if (e.residual.data) {
        get4(e.residual.data, e.residual.f32, o_res + i, n, f);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] += f[u];
    }
    put4(e.out.data, e.out.f32, o_out + i, n, v);
}

// ---- operands ----

// Eight floats as three planes of bfloat16; what is infinite or NaN lies in the first alone (as does what bfloat16
// rounds to infinity, from 3.39e38 on).
__device__ inline void cut(const float (&f)[8], uint4 (&plane)[3])
{
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    uint32_t *h = reinterpret_cast<uint32_t *>(&plane[0]), *m = reinterpret_cast<uint32_t *>(&plane[1]),
             *l = reinterpret_cast<uint32_t *>(&plane[2]);
    auto both = [](float a, float b) {
        return __builtin_bit_cast(uint32_t, (pair{static_cast<__bf16>(a), static_cast<__bf16>(b)}));
    };
    auto low = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto high = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
    const float inf = __builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = both(f[2 * i], f[2 * i + 1]);
        float a = fabsf(low(h[i])) < inf ? f[2 * i] - low(h[i]) : 0.f;
        float b = fabsf(high(h[i])) < inf ? f[2 * i + 1] - high(h[i]) : 0.f;
        m[i] = both(a, b);
        l[i] = both(a - low(m[i]), b - high(m[i]));
    }
}

template <typename T>
constexpr int PLANES = sizeof(T) == 4 ? 3 : 1;
constexpr int LDS_PAD = 4;  // rows between the chunks of 8 of k: 16 lanes that store 4 rows of 4 chunks hit all banks

// The X rows' (or columns') share of one step: BX of them by BK of k, in units of 8 of k of one row (along k), or of two
// columns (across k).
template <typename T, bool ACROSS, int BX, int BK, int NTB>
struct Stage {
    static constexpr int CH = BK / 8, PITCH = BX + LDS_PAD;
    static constexpr int UNITS = ACROSS ? BX / 2 * CH : BX * CH;
    static constexpr int U = (UNITS + NTB - 1) / NTB;
    static constexpr int LDS = PLANES<T> * CH * PITCH;  // vectors of 16 bytes
    typedef typename Vec<T>::raw raw;
    typedef typename Vec<T>::mem mem;
    static constexpr int PARTS = 8 / Vec<T>::N;

    raw x[U][ACROSS ? 1 : PARTS];       // along k
    uint32_t y[U][ACROSS ? 8 : 1][ACROSS ? PARTS : 1];  // across k: two columns in a word, or in two
    const T *row[U];
    int x0, X;

    __device__ static int unit(int u) { return u * NTB + static_cast<int>(threadIdx.x); }
    __device__ static bool any(int u) { return UNITS % NTB == 0 || unit(u) < UNITS; }

    __device__ void begin(const Mat &m, int at, int n)
    {
        x0 = at, X = n;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (ACROSS) {
                row[u] = static_cast<const T *>(m.data);
            } else {
                // (rows past the last are that one again: their products go nowhere)
                const int i = x0 + unit(u) / CH;
                row[u] = static_cast<const T *>(m.data) + m.row(i < X ? i : X - 1);
            }
        }
    }
    // k from k0 on; past k1 zeros
    __device__ void load(const Mat &m, int k0, int k1)
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            if constexpr (ACROSS) {
                const int i = x0 + unit(u) % (BX / 2) * 2, k = k0 + unit(u) / (BX / 2) * 8;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if constexpr (PARTS == 2)
                        y[u][r][0] = y[u][r][1] = 0;
                    else
                        y[u][r][0] = 0;
                    if (k + r < k1 && i < X) {
                        const T *p = row[u] + m.row(k + r) + i;
                        if (i + 1 < X) {
                            if constexpr (PARTS == 2) {
                                typedef uint32_t two __attribute__((ext_vector_type(2), aligned(4)));
                                const two w = *reinterpret_cast<const two *>(p);
                                y[u][r][0] = w[0], y[u][r][1] = w[1];
                            } else {
                                typedef uint32_t one __attribute__((aligned(2)));
                                y[u][r][0] = *reinterpret_cast<const one *>(p);
                            }
                        } else {
                            if constexpr (PARTS == 2)
                                y[u][r][0] = __float_as_uint(Vec<T>::one(p));
                            else
                                y[u][r][0] = __float_as_uint(Vec<T>::one(p)) >> 16;
                        }
                    }
                }
            } else {
                const int k = k0 + unit(u) % CH * 8;
                const T *p = row[u] + k;
                if (k + 8 <= k1) {
#pragma unroll
                    for (int v = 0; v < PARTS; ++v)
                        x[u][v] = *reinterpret_cast<const mem *>(p + v * Vec<T>::N);
                } else {
#pragma unroll
                    for (int v = 0; v < PARTS; ++v) {
                        x[u][v] = raw{0, 0, 0, 0};
#pragma unroll
                        for (int e = 0; e < Vec<T>::N; ++e)
                            if (k + v * Vec<T>::N + e < k1)
                                Vec<T>::set(x[u][v], e, Vec<T>::one(p + v * Vec<T>::N + e));
                    }
                }
            }
        }
    }
    __device__ static void put(uint4 *lds, int chunk, int i, const float (&f)[8])
    {
        uint4 plane[3];
        cut(f, plane);
#pragma unroll
        for (int p = 0; p < 3; ++p)
            lds[(p * CH + chunk) * PITCH + i] = plane[p];
    }
    __device__ void store(uint4 *lds) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            if constexpr (ACROSS) {
                const int i = unit(u) % (BX / 2) * 2, chunk = unit(u) / (BX / 2);
                if constexpr (PARTS == 2) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        float f[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            f[r] = __uint_as_float(y[u][r][s]);
                        put(lds, chunk, i + s, f);
                    }
                } else {
                    uint4 a, b;
                    uint32_t *pa = reinterpret_cast<uint32_t *>(&a), *pb = reinterpret_cast<uint32_t *>(&b);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        pa[r] = __builtin_amdgcn_perm(y[u][2 * r + 1][0], y[u][2 * r][0], 0x05040100u);
                        pb[r] = __builtin_amdgcn_perm(y[u][2 * r + 1][0], y[u][2 * r][0], 0x07060302u);
                    }
                    lds[chunk * PITCH + i] = a;
                    lds[chunk * PITCH + i + 1] = b;
                }
            } else {
                const int chunk = unit(u) % CH, i = unit(u) / CH;
                if constexpr (PARTS == 2) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = x[u][e / 4][e % 4];
                    put(lds, chunk, i, f);
                } else {
                    lds[chunk * PITCH + i] = __builtin_bit_cast(uint4, x[u][0]);
                }
            }
        }
    }
    // The lane's 8 of k (step kk of 32) of row i of a plane.
    __device__ static bf16x8 fragment(const uint4 *lds, int plane, int kk, int i)
    {
        const int lane = threadIdx.x & 63;
        return __builtin_bit_cast(bf16x8, lds[(plane * CH + kk * 4 + (lane >> 4)) * PITCH + i + (lane & 15)]);
    }
};

struct Gemm {
    Mat a, b;
    int I, J, K;
    int ti, tj, splits, k_split;  // tiles, parts of k of k_split each
    bool i_inner;                 // tiles that share a j come one after the other (else those that share an i)
    float *partial;               // [splits, J, pitch], where splits > 1
    int pitch;
    Epilogue e;
};

// A launch's blocks go to the 8 dies in turn; the die's own blocks take neighbouring tiles, whose shared operand its
// cache then holds.
__device__ inline int tile_id(int n)
{
    const int die = blockIdx.x & 7, at = blockIdx.x >> 3, per = n >> 3, more = n & 7;
    return die * per + (die < more ? die : more) + at;
}

template <typename TA, typename TB, bool A_ACROSS, bool B_ACROSS, int BI, int BJ, int WI, int WJ, int BK>
__global__ __launch_bounds__(BI / WI * (BJ / WJ) * 64) void k_gemm(Gemm g)
{
    constexpr int NTB = BI / WI * (BJ / WJ) * 64;
    typedef Stage<TA, A_ACROSS, BI, BK, NTB> SA;
    typedef Stage<TB, B_ACROSS, BJ, BK, NTB> SB;
    constexpr int FI = WI / 16, FJ = WJ / 16, PA = PLANES<TA>, PB = PLANES<TB>;
    __shared__ uint4 lds[SA::LDS + SB::LDS];
    const int tiles = g.ti * g.tj, id = tile_id(tiles * g.splits);
    const int split = id / tiles, tile = id - split * tiles;
    const int outer = g.i_inner ? tile / g.ti : tile / g.tj, inner = tile - outer * (g.i_inner ? g.ti : g.tj);
    const int i0 = (g.i_inner ? inner : outer) * BI, j0 = (g.i_inner ? outer : inner) * BJ;
    const int k0 = split * g.k_split, k1 = k0 + g.k_split < g.K ? k0 + g.k_split : g.K;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wi = wave % (BI / WI) * WI, wj = wave / (BI / WI) * WJ;
    SA sa;
    SB sb;
    sa.begin(g.a, i0, g.I);
    sb.begin(g.b, j0, g.J);
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int a = 0; a < FI; ++a)
#pragma unroll
        for (int b = 0; b < FJ; ++b)
            acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (k0 < k1) {
        sa.load(g.a, k0, k1);
        sb.load(g.b, k0, k1);
    }
    for (int k = k0; k < k1; k += BK) {
        __syncthreads();
        sa.store(lds);
        sb.store(lds + SA::LDS);
        __syncthreads();
        if (k + BK < k1) {
            sa.load(g.a, k + BK, k1);
            sb.load(g.b, k + BK, k1);
        }
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            bf16x8 fb[PB][FJ];
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int b = 0; b < FJ; ++b)
                    fb[p][b] = SB::fragment(lds + SA::LDS, p, kk, wj + 16 * b);
#pragma unroll
            for (int a = 0; a < FI; ++a) {
                bf16x8 fa[PA];
#pragma unroll
                for (int p = 0; p < PA; ++p)
                    fa[p] = SA::fragment(lds, p, kk, wi + 16 * a);
#pragma unroll
                for (int s = 2; s >= 0; --s)  // (small products first)
#pragma unroll
                    for (int p = 0; p < PA; ++p)
                        if (s - p >= 0 && s - p < PB)
#pragma unroll
                            for (int b = 0; b < FJ; ++b)
                                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[p], fb[s - p < 0 || s - p >= PB ? 0 : s - p][b],
                                                                                   acc[a][b], 0, 0, 0);
            }
        }
    }
    // a lane has four neighbouring i of one j
#pragma unroll
    for (int b = 0; b < FJ; ++b) {
        const int j = j0 + wj + 16 * b + (lane & 15);
        if (j >= g.J)
            continue;
        int64_t o_out = 0, o_pre = 0, o_res = 0;
        if (g.splits > 1) {
            o_out = (static_cast<int64_t>(split) * g.J + j) * g.pitch;
        } else {
            o_out = g.e.out.row(j);
            if (g.e.pre.data)
                o_pre = g.e.pre.row(j);
            if (g.e.residual.data)
                o_res = g.e.residual.row(j);
        }
#pragma unroll
        for (int a = 0; a < FI; ++a) {
            const int i = i0 + wi + 16 * a + 4 * (lane >> 4);
            if (i >= g.I)
                continue;
            if (g.splits > 1) {
                *reinterpret_cast<f32x4 *>(g.partial + o_out + i) = acc[a][b];
            } else {
                float v[4] = {acc[a][b][0], acc[a][b][1], acc[a][b][2], acc[a][b][3]};
                emit(g.e, i, g.I, o_out, o_pre, o_res, v);
            }
        }
    }
}

// Launches of one arrangement of the operands: the tile sizes of `shape` (dhlinear::Shape).
template <typename TA, typename TB, bool A_ACROSS, bool B_ACROSS>
inline hipError_t launch_types(const Gemm &g, int shape, hipStream_t st)
{
    constexpr int BK = sizeof(TA) == 2 && sizeof(TB) == 2 ? 64 : 32;
    const dim3 grid(static_cast<unsigned>(g.ti) * g.tj * g.splits);
    if (shape == dhlinear::LARGE)
        hipLaunchKernelGGL((k_gemm<TA, TB, A_ACROSS, B_ACROSS, 128, 128, 64, 64, BK>), grid, dim3(256), 0, st, g);
    else if (shape == dhlinear::MEDIUM)
        hipLaunchKernelGGL((k_gemm<TA, TB, A_ACROSS, B_ACROSS, 64, 64, 32, 32, BK>), grid, dim3(256), 0, st, g);
    else
        hipLaunchKernelGGL((k_gemm<TA, TB, A_ACROSS, B_ACROSS, 64, 16, 16, 16, BK>), grid, dim3(256), 0, st, g);
    return hipGetLastError();
}

template <bool A_ACROSS, bool B_ACROSS>
inline hipError_t launch_gemm(const Gemm &g, int shape, hipStream_t st)
{
    if (g.a.f32)
        return g.b.f32 ? launch_types<float, float, A_ACROSS, B_ACROSS>(g, shape, st)
                       : launch_types<float, bf16s, A_ACROSS, B_ACROSS>(g, shape, st);
    return g.b.f32 ? launch_types<bf16s, float, A_ACROSS, B_ACROSS>(g, shape, st)
                   : launch_types<bf16s, bf16s, A_ACROSS, B_ACROSS>(g, shape, st);
}

}  // namespace DH_NS
