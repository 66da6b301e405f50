// Products of rows on the matrix cores, with an epilogue: D[j][i] = sum_k A(i, k) B(j, k), the kernels of domino_linear.
//
// An operand lies along k (its row i holds k = 0, 1, ...: x and w of a forward pass) or across k (its row k holds
// i = 0, 1, ...: w where the sum goes over its rows, both where it goes over the batch).  A block takes a tile of
// BI x BJ and BK of k at a time: global memory -> registers (the next step's while this one is multiplied) -> LDS as
// bfloat16, transposed where the operand lies across k, -> v_mfma_f32_16x16x32_bf16, summed in float32.
//
// float32 operands are cut into three bfloat16 planes, x = h + m + l, each the rounded remainder of those before: that
// is all of x's 24 bits (|m| <= 2^-8 |x|, |l| <= 2^-17 |x|), and every product of two planes is exact in float32.  A
// float32 and a bfloat16 operand take 3 products, two float32 operands the 6 without m l, l m and l l, which are at most
// 2^-25, 2^-25 and 2^-34 of the whole product, 2^-24 together.  4096 x 4096 x 4096: 401 us (0.34 PFLOP/s) and 667 us (0.21);
// the library's float32 product takes 920.
//
// What bounds it, on one MI355X.
//   512 x 256 -> 151936 logits with a residual, bfloat16 to float32 (700 MB): 148 us, 4.7 TB/s: HBM, in tiles of 128 x 128
//     whose epilogue goes through LDS, so that rows are read and written in whole lines.
//   16 x 256 -> 151936 (97 MB): 20 us, 4.8 TB/s: HBM.  512 x 5120 -> 256: 9 us in 10 parts, then a join: latency.
//   Gradients of the 512 x 256 x 151936 layer: x's 75 us, 532 TFLOP/s, 320 MB read and written (4.3 TB/s), in 64 parts of
//     8 tiles, and 8.5 for their join; w's 96 us, 414 TFLOP/s, 317 MB (3.3 TB/s).  Both are short of the bytes' time: a
//     step of 64 takes about as long to bring a tile's operands from L2 to LDS as its matrix instructions take.
//   The same layer in float32 (6 products): 264 us, gradients 237 and 254, in tiles of 128 x 128 with one LDS buffer, 0.15 to
//     0.17 PFLOP/s: loads and the cut into planes, which every tile that shares an operand does again.
//   4096 x 4096 x 4096, bfloat16: 124 to 130 us, 1.06 to 1.1 PFLOP/s in tiles of 256 x 256, 183 us in those of 128 x 128;
//     gradients 135 and 150 us.
// Tried and left: rows of LDS that change places by their chunk instead of lying LDS_PAD apart (x's gradient 3% less, that
// of 4096^3 8% more); 3 blocks a compute unit in tiles of 128 x 128 (registers spill: 196, 102 and 180 us for the three
// products of the 512 rows); tiles of 256 x 128 (w's gradient 141 us).
#pragma once

#include "dh_linear.h"
#include "dh_rows.h"

#include <type_traits>

namespace DH_NS {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Rows at data + b bs + r rs, row b R + r; flat: all rs apart.
struct Mat {
    const void *data;
    int64_t bs, rs;
    Divisor by;  // R
    bool flat, near, f32;
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
    // (the rows of a tile within 31 bits, or all of them)
    const int64_t span = (m.B - 1) * m.batch_stride + (m.R - 1) * m.row_stride + m.V;
    t.near = t.flat ? t.rs < (1 << 21) : span < (1 << 29);
    return t;
}

// ---- epilogue ----

// Activations of a few instructions, which a product's epilogue has in every element's place.  gelu's erfc has some
// hundreds, and is in the kernel that joins partial sums alone: all sums go there in float32, 512 x 256 -> 151936 in
// bfloat16 takes 237 us with gelu and 96 with silu, 512 x 1024 -> 4096 25 and 19.
__device__ inline float light_act(float a, int act)
{
    if (act == DOMINO_SILU)
        return a * sigmoidf_(a);
    return act == DOMINO_RELU ? (a > 0.f || a != a ? a : 0.f) : a;
}
__device__ inline float act_of(float a, int act)
{
    if (act == DOMINO_GELU)
        return 0.5f * a * erfcf(-0.70710678f * a);
    return light_act(a, act);
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
template <bool STREAM = false, typename F>
__device__ inline void get4(const void *data, bool f32, int64_t o, int n, F &f)
{
    if (f32) {
        const float *p = static_cast<const float *>(data) + o;
        if (n >= 4) {
            const auto *v = reinterpret_cast<const Vec<float>::mem *>(p);
            const Vec<float>::raw x = STREAM ? __builtin_nontemporal_load(v) : *v;
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
            const auto *v = reinterpret_cast<const two *>(p);
            const two x = STREAM ? __builtin_nontemporal_load(v) : *v;
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
template <bool STREAM = false, typename F>
__device__ inline void put4(const void *data, bool f32, int64_t o, int n, const F &f)
{
    if (f32) {
        float *p = static_cast<float *>(const_cast<void *>(data)) + o;
        if (n >= 4) {
            const Vec<float>::raw x = {f[0], f[1], f[2], f[3]};
            if (STREAM)
                __builtin_nontemporal_store(x, reinterpret_cast<Vec<float>::mem *>(p));
            else
                *reinterpret_cast<Vec<float>::mem *>(p) = x;
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
            const two x = {Vec<bf16s>::bits(f[0]) | (Vec<bf16s>::bits(f[1]) << 16),
                           Vec<bf16s>::bits(f[2]) | (Vec<bf16s>::bits(f[3]) << 16)};
            if (STREAM)
                __builtin_nontemporal_store(x, reinterpret_cast<two *>(p));
            else
                *reinterpret_cast<two *>(p) = x;
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
    bool bias_f32, stream;   // stream: out and residual are too large for the caches
    int act;
};

// Elements i .. i + 3 (those below I) of row j.  GELU: any activation, else a light one.
template <bool GELU>
__device__ inline void emit(const Epilogue &e, int i, int I, int64_t o_out, int64_t o_pre, int64_t o_res, f32x4 v)
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
            v[u] = GELU ? act_of(v[u], e.act) : light_act(v[u], e.act);
    if (e.residual.data) {
        get4(e.residual.data, e.residual.f32, o_res + i, n, f);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] += f[u];
    }
    put4(e.out.data, e.out.f32, o_out + i, n, v);
}

// The same for a block's tile of BI x BJ from (i0, j0), with a light activation, by way of LDS (`tile`, free after a
// barrier), PART rows at a time: a thread has the elements i .. i + 3 of every STEP-th row, so that a row's neighbours are
// loaded and stored together.  The residual is on its way before the sums are exchanged.
template <int BI, int BJ, int NTB>
struct EmitTile {
    static constexpr int PART = BJ < 64 ? BJ : 64;
    static constexpr int LANES = BI / 4, STEP = NTB / LANES, N = PART / STEP, PITCH = BI + 4;
    static constexpr int LDS = PART * PITCH / 4;  // vectors of 16 bytes
    static constexpr int G = N < 8 ? N : 8;       // rows in registers at once
    static_assert(PART % STEP == 0 && N % G == 0 && BJ % PART == 0, "");

    template <bool F32, bool STREAM>
    __device__ static void get(const Mat &m, int i, int j0, int J, f32x4 (&v)[G])
    {
#pragma unroll
        for (int u = 0; u < G; ++u) {
            const int j = j0 + u * STEP;
            get4<STREAM>(m.data, F32, m.row(j < J ? j : J - 1) + i, 4, v[u]);
        }
    }
    template <bool F32, bool STREAM>
    __device__ static void put(const Mat &m, int i, int j0, int J, const f32x4 (&v)[G])
    {
#pragma unroll
        for (int u = 0; u < G; ++u) {
            const int j = j0 + u * STEP;
            if (j < J)
                put4<STREAM>(m.data, F32, m.row(j) + i, 4, v[u]);
        }
    }

    // store(tile): the waves that hold the rows from j0 on write them to rows of PITCH floats.
    template <typename STORE>
    __device__ static void part(const Epilogue &e, int i0, int I, int j0, int J, float *tile, STORE store)
    {
        const int c = 4 * (static_cast<int>(threadIdx.x) % LANES), r = static_cast<int>(threadIdx.x) / LANES, i = i0 + c;
        const bool whole = i + 4 <= I;
        const float *mine = tile + r * PITCH + c;
        f32x4 bias = {0.f, 0.f, 0.f, 0.f}, res[G];
        j0 += r;
        const auto residual = [&](int j) {
            if (e.residual.f32)
                e.stream ? get<true, true>(e.residual, i, j, J, res) : get<true, false>(e.residual, i, j, J, res);
            else
                e.stream ? get<false, true>(e.residual, i, j, J, res) : get<false, false>(e.residual, i, j, J, res);
        };
        if (whole && e.residual.data)
            residual(j0);
        if (whole && e.bias)
            get4(e.bias, e.bias_f32, i, 4, bias);
        __syncthreads();
        store(tile);
        __syncthreads();
        if (!whole) {
#pragma unroll 1
            for (int u = 0; i < I && u < N && j0 + u * STEP < J; ++u) {
                const int j = j0 + u * STEP;
                emit<false>(e, i, I, e.out.row(j), e.pre.data ? e.pre.row(j) : 0, e.residual.data ? e.residual.row(j) : 0,
                     *reinterpret_cast<const f32x4 *>(mine + u * STEP * PITCH));
            }
            return;
        }
#pragma unroll 1
        for (int u0 = 0; u0 < N; u0 += G, j0 += G * STEP, mine += G * STEP * PITCH) {
            f32x4 v[G];
            if (u0 && e.residual.data)
                residual(j0);
#pragma unroll
            for (int u = 0; u < G; ++u)
                v[u] = *reinterpret_cast<const f32x4 *>(mine + u * STEP * PITCH) + bias;
            if (e.pre.data) {
                if (e.pre.f32)
                    put<true, false>(e.pre, i, j0, J, v);
                else
                    put<false, false>(e.pre, i, j0, J, v);
            }
            const auto activate = [&](int act) {
#pragma unroll
                for (int u = 0; u < G; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[u][k] = light_act(v[u][k], act);
            };
            if (e.act == DOMINO_SILU)
                activate(DOMINO_SILU);
            else if (e.act == DOMINO_RELU)
                activate(DOMINO_RELU);
            if (e.residual.data) {
#pragma unroll
                for (int u = 0; u < G; ++u)
                    v[u] += res[u];
            }
            if (e.out.f32)
                e.stream ? put<true, true>(e.out, i, j0, J, v) : put<true, false>(e.out, i, j0, J, v);
            else
                e.stream ? put<false, true>(e.out, i, j0, J, v) : put<false, false>(e.out, i, j0, J, v);
        }
    }
};

// ---- operands ----

// Eight floats as three planes of bfloat16.  The first is cut off at bfloat16's largest value, past which finite floats
// would round to infinity; of an infinity or NaN the planes are such, or NaN, so that their products are not finite.
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
    const float most = __uint_as_float(0x7F7F0000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = both(__builtin_amdgcn_fmed3f(f[2 * i], -most, most), __builtin_amdgcn_fmed3f(f[2 * i + 1], -most, most));
        const float a = f[2 * i] - low(h[i]), b = f[2 * i + 1] - high(h[i]);
        m[i] = both(a, b);
        l[i] = both(a - low(m[i]), b - high(m[i]));
    }
}
// Two floats as what they make of a product with an infinity: infinities and NaN as they are, any other cut off to
// bfloat16, but none to 0 (nor to a number that counts as one) that is not 0.
__device__ inline uint32_t kinds(float a, float b)
{
    const auto one = [](float f) {
        const uint32_t w = __float_as_uint(f), size = w & 0x7FFFFFFFu;
        return size > 0x7F800000u ? 0x7FC0u : size && size < 0x00800000u ? (w >> 16 & 0x8000u) | 0x80u : w >> 16;
    };
    return one(a) | one(b) << 16;
}

template <typename T>
constexpr int PLANES = sizeof(T) == 4 ? 3 : 1;
constexpr int LDS_PAD = 2;  // rows between the chunks of 8 of k, so that 8 lanes that store a row's chunks hit all banks

// The X rows' (or columns') share of one step: BX of them by BK of k, in units of 8 of k of one row (along k), or of 8 of
// k of the columns that 8 bytes hold (across k).  near: the addresses of a tile are a common one and 32 bits.
// D: steps that are in registers at once.
template <typename T, bool ACROSS, int BX, int BK, int NTB, int D>
struct Stage {
    static constexpr int CH = BK / 8, PITCH = BX + LDS_PAD, SIZE = sizeof(T);
    static constexpr int COLS = 8 / SIZE;
    static constexpr int UNITS = ACROSS ? BX / COLS * CH : BX * CH;
    static constexpr int U = (UNITS + NTB - 1) / NTB;
    static constexpr int LDS = PLANES<T> * CH * PITCH;  // vectors of 16 bytes
    static constexpr int PARTS = 8 / Vec<T>::N;
    typedef typename Vec<T>::raw raw;
    typedef typename Vec<T>::mem mem;
    typedef uint32_t two __attribute__((ext_vector_type(2)));
    typedef uint32_t two_mem __attribute__((ext_vector_type(2), aligned(2)));

    raw x[D][ACROSS ? 1 : U][PARTS];
    two y[D][ACROSS ? U : 1][8];
    uint32_t off[U];
    const char *base;  // of the tile's first row and k = 0
    int64_t step;      // bytes from a k to the next
    int x0, X;
    int end;  // across k: the tile's column where the operand's last whole unit begins (negative in a tile of a few columns)
    bool fast;

    __device__ static int unit(int u) { return u * NTB + static_cast<int>(threadIdx.x); }
    __device__ static bool any(int u) { return UNITS % NTB == 0 || unit(u) < UNITS; }
    // The first column of a unit.  Those that reach past the operand's last column take its last whole unit, once more.
    __device__ int column(int u) const
    {
        const int i = unit(u) % (BX / COLS) * COLS;
        return i < end ? i : end;
    }
    __device__ static int place(int i) { return ACROSS ? i ^ ((i >> 4) & 3) : i; }  // (4 columns a lane: all banks again)

    __device__ void begin(const Mat &m, int at, int n)
    {
        x0 = at, X = n;
        const char *data = static_cast<const char *>(m.data);
        // (rows past the last are that one again, columns past it whatever LDS holds: their products go nowhere)
        end = X - COLS - x0;
        fast = m.near && !(ACROSS && (X < COLS || !m.flat));
        const int before = end < 0 ? -end : 0;
        if constexpr (ACROSS) {
            base = data + (static_cast<int64_t>(x0) - before) * SIZE;
            step = m.rs * SIZE;
        } else {
            base = m.flat ? data + static_cast<int64_t>(x0) * m.rs * SIZE : data;
            step = SIZE;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (ACROSS) {
                off[u] = static_cast<uint32_t>(unit(u) / (BX / COLS) * 8 * static_cast<uint32_t>(step) +
                                               (column(u) + before) * SIZE);
            } else {
                const int last = X - 1 - x0, i = unit(u) / CH < last ? unit(u) / CH : last;
                off[u] = (m.flat ? static_cast<uint32_t>(i) * static_cast<uint32_t>(m.rs * SIZE)
                                 : static_cast<uint32_t>(m.row(x0 + i) * SIZE)) + unit(u) % CH * 8 * SIZE;
            }
        }
    }
    // A whole step's share, k from k0 on, into registers: the short way.
    template <int S>
    __device__ void load(int k0)
    {
        const char *from = base + k0 * step;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            if constexpr (ACROSS) {
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    y[S][u][r] = *reinterpret_cast<const two_mem *>(
                        from + static_cast<uint32_t>(off[u] + r * static_cast<uint32_t>(step)));
            } else {
#pragma unroll
                for (int v = 0; v < PARTS; ++v)
                    x[S][u][v] = *reinterpret_cast<const mem *>(from + off[u] + 16 * v);
            }
        }
    }
    // The last of k, fewer than a step's: rows past it are that row again, and become zeros.
    __device__ void load_last(int k0, int k1)
    {
        const char *from = base + k0 * step;
        const int left = k1 - 1 - k0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = unit(u) / (BX / COLS) * 8, column_off = static_cast<int>(off[u] - k * static_cast<uint32_t>(step));
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int at = k + r < left ? k + r : left;
                y[0][u][r] = two{0, 0};
                if (any(u))
                    y[0][u][r] = *reinterpret_cast<const two_mem *>(
                        from + static_cast<uint32_t>(column_off + at * static_cast<uint32_t>(step)));
            }
#pragma unroll
            for (int r = 0; r < 8; ++r)
                y[0][u][r] = k + r <= left ? y[0][u][r] : two{0, 0};
        }
    }
    // Any strides, edges and ends: k from k0 on, past k1 zeros, to LDS.  KIND: the elements' kinds(), as one plane.
    template <bool KIND = false>
    __device__ void slow(const Mat &m, int k0, int k1, uint4 *lds)
    {
        if constexpr (ACROSS && !KIND)
            if (fast) {
                load_last(k0, k1);
                store<0>(lds);
                return;
            }
        const T *data = static_cast<const T *>(m.data);
#pragma unroll 1
        for (int q = threadIdx.x; q < BX * CH; q += NTB) {
            const int row = ACROSS ? q % BX : q / CH, chunk = ACROSS ? q / BX : q % CH, k = k0 + 8 * chunk;
            const int i = x0 + row < X ? x0 + row : X - 1;
            const T *p = ACROSS ? data + i : data + m.row(i);
            float f[8];
            // (loads without conditions are in flight together; past the end, the last one again)
            const int last = k1 - 1 - k;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int at = k + (r < last ? r : last);
                f[r] = Vec<T>::one(ACROSS ? p + m.row(at) : p + at);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r)
                f[r] = r <= last ? f[r] : 0.f;
            if constexpr (SIZE == 4 && !KIND) {
                put(lds, chunk, row, f);
            } else {
                uint4 w;
                uint32_t *pw = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    pw[r] = KIND ? kinds(f[2 * r], f[2 * r + 1])
                                 : (__float_as_uint(f[2 * r]) >> 16) | (__float_as_uint(f[2 * r + 1]) & 0xFFFF0000u);
                lds[chunk * PITCH + place(row)] = w;
            }
        }
    }
    __device__ static void put(uint4 *lds, int chunk, int i, const float (&f)[8])
    {
        uint4 plane[3];
        cut(f, plane);
#pragma unroll
        for (int p = 0; p < 3; ++p)
            lds[(p * CH + chunk) * PITCH + place(i)] = plane[p];
    }
    // What load() took, to LDS.
    template <int S>
    __device__ void store(uint4 *lds) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            if constexpr (ACROSS) {
                const int i = column(u), chunk = unit(u) / (BX / COLS);
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const int at = (i + c) & (BX - 1);  // (those before the tile go behind its last column)
                    if constexpr (SIZE == 4) {
                        float f[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            f[r] = __uint_as_float(y[S][u][r][c]);
                        put(lds, chunk, at, f);
                    } else {
                        uint4 w;
                        uint32_t *pw = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            pw[r] = __builtin_amdgcn_perm(y[S][u][2 * r + 1][c >> 1], y[S][u][2 * r][c >> 1],
                                                          c & 1 ? 0x07060302u : 0x05040100u);
                        lds[chunk * PITCH + place(at)] = w;
                    }
                }
            } else {
                const int chunk = unit(u) % CH, i = unit(u) / CH;
                if constexpr (PARTS == 2) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = x[S][u][e / 4][e % 4];
                    put(lds, chunk, i, f);
                } else {
                    lds[chunk * PITCH + i] = __builtin_bit_cast(uint4, x[S][u][0]);
                }
            }
        }
    }
    // The lane's 8 of k (step kk of 32) of row i + lane % 16 of a plane; i a multiple of 16.
    __device__ static bf16x8 fragment(const uint4 *lds, int plane, int kk, int i)
    {
        const int lane = threadIdx.x & 63;
        return __builtin_bit_cast(bf16x8, lds[(plane * CH + kk * 4 + (lane >> 4)) * PITCH + place(i + (lane & 15))]);
    }
};

struct Gemm {
    Mat a, b;
    int I, J, K;
    int ti, tj, splits;           // tiles; parts of k: part p takes the steps p, p + splits, p + 2 splits, ...
    bool i_inner;                 // tiles that share a j come one after the other (else those that share an i)
    float *partial;               // [splits, J, pitch], or NULL: the results go out (splits = 1)
    int pitch;
    Epilogue e;
};

// Waves a SIMD that a kernel's registers allow.
template <typename TA, typename TB, int ACROSS, int TILE>
constexpr int WAVES = TILE >= 128 * 128 || ACROSS == 2 ? 2 : sizeof(TA) == 2 && sizeof(TB) == 2 && !ACROSS ? 4 : 3;

// A launch's blocks go to the 8 dies in turn; the die's own blocks take neighbouring tiles, whose shared operand its
// cache then holds.
__device__ inline int tile_id(int block, int n)
{
    const int die = block & 7, at = block >> 3, per = n >> 3, more = n & 7;
    return die * per + (die < more ? die : more) + at;
}

// One of a product's tiles, by a block.
template <typename TA, typename TB, bool A_ACROSS, bool B_ACROSS, int BI, int BJ, int WI, int WJ, int BK>
struct Tile {
    static constexpr int NTB = BI / WI * (BJ / WJ) * 64;
    // (two steps ahead of the one that is multiplied, where the registers allow it)
    static constexpr int D = sizeof(TA) == 2 && sizeof(TB) == 2 && BI * BJ <= 128 * 128 ? 2 : 1;
    typedef Stage<TA, A_ACROSS, BI, BK, NTB, D> SA;
    typedef Stage<TB, B_ACROSS, BJ, BK, NTB, D> SB;
    typedef EmitTile<BI, BJ, NTB> Emit;
    static constexpr int LDS = SA::LDS + SB::LDS, BUF = LDS * 32 <= (NTB == 256 ? 80 << 10 : 160 << 10) ? 2 : 1;
    static constexpr int LDS_ALL = BUF * LDS > Emit::LDS ? BUF * LDS : Emit::LDS;  // vectors of 16 bytes

    __device__ static void run(const Gemm &g, int block, uint4 *lds);
};

template <typename TA, typename TB, bool A_ACROSS, bool B_ACROSS, int BI, int BJ, int WI, int WJ, int BK>
__device__ __forceinline__ void Tile<TA, TB, A_ACROSS, B_ACROSS, BI, BJ, WI, WJ, BK>::run(const Gemm &g, int block,
                                                                                        uint4 *lds)
{
    constexpr int FI = WI / 16, FJ = WJ / 16, PA = PLANES<TA>, PB = PLANES<TB>;
    const int tiles = g.ti * g.tj, id = tile_id(block, tiles * g.splits);
    const int split = id / tiles, tile = id - split * tiles;
    const int outer = g.i_inner ? tile / g.ti : tile / g.tj, inner = tile - outer * (g.i_inner ? g.ti : g.tj);
    const int i0 = (g.i_inner ? inner : outer) * BI, j0 = (g.i_inner ? outer : inner) * BJ;
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
    uint4 *at = lds;
    const auto multiply = [&]() {
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            bf16x8 fb[PB][FJ];
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int b = 0; b < FJ; ++b)
                    fb[p][b] = SB::fragment(at + SA::LDS, p, kk, wj + 16 * b);
#pragma unroll
            for (int a = 0; a < FI; ++a) {
                bf16x8 fa[PA];
#pragma unroll
                for (int p = 0; p < PA; ++p)
                    fa[p] = SA::fragment(at, p, kk, wi + 16 * a);
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
        if constexpr (BUF == 2)
            at = at == lds ? lds + LDS : lds;
    };
    // whole steps, without a condition between the loads and their use: the wait for a step's loads leaves those of the
    // next step in flight
    const int steps = sa.fast && sb.fast ? g.K / BK : 0, every = (g.K + BK - 1) / BK;
    const int last = steps - 1;
    const auto load = [&](auto slot, int t) {
        constexpr int S = decltype(slot)::value;
        t = t < last ? t : last;  // (past the last one: that one, for nothing)
        sa.template load<S>(t * BK);
        sb.template load<S>(t * BK);
        __builtin_amdgcn_sched_barrier(0);  // (they go out now, not where they are used)
    };
    const auto step = [&](auto slot, int t) {
        constexpr int S = decltype(slot)::value;
        // (of two buffers, the one of the last step but one: all waves are past it once they have met in the last step)
        if constexpr (BUF == 1)
            __syncthreads();
        sa.template store<S>(at);
        sb.template store<S>(at + SA::LDS);
        __syncthreads();
        load(slot, t + D * g.splits);
        multiply();
    };
    typedef std::integral_constant<int, 0> First;
    typedef std::integral_constant<int, D - 1> Second;
    int t = split;
    if (t < steps) {
        load(First{}, t);
        if constexpr (D == 2) {
            load(Second{}, t + g.splits);
            for (; t + g.splits < steps; t += 2 * g.splits) {
                step(First{}, t);
                step(Second{}, t + g.splits);
            }
        }
        for (; t < steps; t += g.splits)  // (with two in registers: one at the most)
            step(First{}, t);
    }
    for (; t < every; t += g.splits) {
        if constexpr (BUF == 1)
            __syncthreads();
        sa.slow(g.a, t * BK, g.K, at);
        sb.slow(g.b, t * BK, g.K, at + SA::LDS);
        __syncthreads();
        multiply();
    }
    // Planes of 0 make NaN of an infinity's other products, and parts of an overflowing product can have both signs.  Where
    // a sum of planes is not finite, the operands' kinds say whether, and with what sign, the product's is: a tile that
    // has one (0 for each finite sum: one more barrier) takes its sum once more in one plane (512 x 256 -> 151936 in
    // float32: 263 us, with a NaN in every row 766).
    if constexpr (PA + PB > 2) {
        const int i = i0 + wi + 4 * (lane >> 4), j = j0 + wj + (lane & 15);
        float odd = 0.f;
#pragma unroll
        for (int a = 0; a < FI; ++a)
#pragma unroll
            for (int b = 0; b < FJ; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)  // (columns past an operand's last are whatever LDS held)
                    if ((!A_ACROSS || i + 16 * a + e < g.I) && (!B_ACROSS || j + 16 * b < g.J))
                        odd = fmaf(acc[a][b][e], 0.f, odd);
        if (__syncthreads_or(odd != odd)) {
            f32x4 kind[FI][FJ];
#pragma unroll
            for (int a = 0; a < FI; ++a)
#pragma unroll
                for (int b = 0; b < FJ; ++b)
                    kind[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int s = split; s < every; s += g.splits) {
                __syncthreads();
                sa.template slow<true>(g.a, s * BK, g.K, lds);
                sb.template slow<true>(g.b, s * BK, g.K, lds + SA::LDS);
                __syncthreads();
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)
#pragma unroll
                    for (int a = 0; a < FI; ++a)
#pragma unroll
                        for (int b = 0; b < FJ; ++b)
                            kind[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                SA::fragment(lds, 0, kk, wi + 16 * a), SB::fragment(lds + SA::LDS, 0, kk, wj + 16 * b),
                                kind[a][b], 0, 0, 0);
            }
            const float inf = __builtin_huge_valf();
#pragma unroll
            for (int a = 0; a < FI; ++a)
#pragma unroll
                for (int b = 0; b < FJ; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[a][b][e] = fabsf(acc[a][b][e]) < inf || fabsf(kind[a][b][e]) < inf ? acc[a][b][e] : kind[a][b][e];
        }
    }
    // a lane has four neighbouring i of one j
    if (!g.partial) {
        static_assert(Emit::PART % WJ == 0, "a wave's rows are in one part");
#pragma unroll 1
        for (int p = 0; p < BJ; p += Emit::PART)
            Emit::part(g.e, i0, g.I, j0 + p, g.J, reinterpret_cast<float *>(lds), [&](float *tile) {
                if (wj < p || wj >= p + Emit::PART)
                    return;
#pragma unroll
                for (int b = 0; b < FJ; ++b)
#pragma unroll
                    for (int a = 0; a < FI; ++a)
                        *reinterpret_cast<f32x4 *>(tile + (wj - p + 16 * b + (lane & 15)) * Emit::PITCH + wi + 16 * a +
                                                   4 * (lane >> 4)) = acc[a][b];
            });
        return;
    }
#pragma unroll
    for (int b = 0; b < FJ; ++b) {
        const int j = j0 + wj + 16 * b + (lane & 15);
        float *part = g.partial + (static_cast<int64_t>(split) * g.J + j) * g.pitch;
        if (j < g.J)
#pragma unroll
            for (int a = 0; a < FI; ++a) {
                const int i = i0 + wi + 16 * a + 4 * (lane >> 4);
                if (i < g.I)
                    *reinterpret_cast<f32x4 *>(part + i) = acc[a][b];
            }
    }
}

template <typename TA, typename TB, bool A_ACROSS, bool B_ACROSS, int BI, int BJ, int WI, int WJ, int BK>
__global__ __launch_bounds__(BI / WI * (BJ / WJ) * 64, (WAVES<TA, TB, A_ACROSS + B_ACROSS, BI * BJ>)) void k_gemm(Gemm g)
{
    typedef Tile<TA, TB, A_ACROSS, B_ACROSS, BI, BJ, WI, WJ, BK> T;
    __shared__ uint4 lds[T::LDS_ALL];
    T::run(g, static_cast<int>(blockIdx.x), lds);
}

template <typename TA, typename TB>
constexpr int STEP_K = sizeof(TA) == 2 && sizeof(TB) == 2 ? 64 : 32;

// Launches of one arrangement of the operands: the tile sizes of `shape` (dhlinear::Shape).
template <typename TA, typename TB, bool A_ACROSS, bool B_ACROSS>
inline hipError_t launch_types(const Gemm &g, int shape, hipStream_t st)
{
    constexpr int BK = STEP_K<TA, TB>;
    const dim3 grid(static_cast<unsigned>(g.ti) * g.tj * g.splits);
    if constexpr (BK == 64)
        if (shape == dhlinear::HUGE) {
            hipLaunchKernelGGL((k_gemm<TA, TB, A_ACROSS, B_ACROSS, 256, 256, 128, 64, BK>), grid, dim3(512), 0, st, g);
            return hipGetLastError();
        }
    if (shape == dhlinear::LARGE)
        hipLaunchKernelGGL((k_gemm<TA, TB, A_ACROSS, B_ACROSS, 128, 128, 64, 64, BK>), grid, dim3(256), 0, st, g);
    else if (shape == dhlinear::MEDIUM)
        hipLaunchKernelGGL((k_gemm<TA, TB, A_ACROSS, B_ACROSS, 64, 64, 32, 32, BK>), grid, dim3(256), 0, st, g);
    else if constexpr (!A_ACROSS)  // (forward)
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
