// Linear layers: y = act(x w^T + bias) + residual, and the gradients of x, w and bias.
//
//     pre = x w^T + bias            y = act(pre) + residual
//     dpre = g act'(pre)            dx = dpre w      dw = dpre^T x      dbias = sum over the rows of dpre
//
// The products are k_gemm's (dh_gemm.h).  Here: how a product is cut into tiles and parts of its sum, the join of
// those parts, and what comes before the backward products (dpre, in float32, and the sums over its rows).
#define DH_NT 256
#define DH_NS dhl
#include "dh_gemm.h"

#include <algorithm>
#include <cmath>

namespace DH_NS {

hipError_t product_y(const Gemm &g, int shape, hipStream_t st);
hipError_t product_dx(const Gemm &g, int shape, hipStream_t st);
hipError_t product_dw(const Gemm &g, int shape, hipStream_t st);
hipError_t product_pair(const Gemm &x, const Gemm &w, hipStream_t st);

// The parts of a product's sums, in order, and the epilogue.  Four elements a thread.
__device__ inline void join_block(const Gemm &g, const Divisor &per, uint32_t block)
{
    const uint32_t at = block * NT + threadIdx.x;
    const int j = static_cast<int>(per.quotient(at)), i = 4 * static_cast<int>(at - j * per.d);
    if (j >= g.J)
        return;
    const int64_t step = static_cast<int64_t>(g.J) * g.pitch;
    const float *p = g.partial + static_cast<int64_t>(j) * g.pitch + i;
    f32x4 sum = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll 8
    for (int s = 1; s < g.splits; ++s)
        sum += *reinterpret_cast<const f32x4 *>(p + s * step);
    emit<true>(g.e, i, g.I, g.e.out.row(j), g.e.pre.data ? g.e.pre.row(j) : 0,
               g.e.residual.data ? g.e.residual.row(j) : 0, sum);
}
__global__ __launch_bounds__(NT) void k_gemm_join(Gemm g, Divisor per) { join_block(g, per, blockIdx.x); }

// The sums of k_dpre's blocks of rows: a wave takes every 4th of them, a lane a column.
struct Bias {
    const float *sums;  // NULL: not wanted
    int blocks, N, N4;
    Mat out;
    bool accumulate;
};
__device__ inline void bias_block(const Bias &b, int block)
{
    __shared__ float part[NWAVE][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = block * 64 + lane;
    float sum = 0.f;
    if (c < b.N)
#pragma unroll 8
        for (int r = wave; r < b.blocks; r += NWAVE)
            sum += b.sums[static_cast<int64_t>(r) * b.N4 + c];
    part[wave][lane] = sum;
    __syncthreads();
    if (wave || c >= b.N)
        return;
    sum = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    if (b.out.f32) {
        float *p = static_cast<float *>(const_cast<void *>(b.out.data)) + c;
        *p = b.accumulate ? *p + sum : sum;
    } else {
        bf16s *p = static_cast<bf16s *>(const_cast<void *>(b.out.data)) + c;
        Vec<bf16s>::put(p, b.accumulate ? Vec<bf16s>::one(p) + sum : sum);
    }
}

// What is to be joined of a backward pass: nx and nw blocks for the products, the others for the bias.
__global__ __launch_bounds__(NT) void k_join(Gemm x, Divisor px, uint32_t nx, Gemm w, Divisor pw, uint32_t nw, Bias b)
{
    if (blockIdx.x < nx)
        join_block(x, px, blockIdx.x);
    else if (blockIdx.x < nx + nw)
        join_block(w, pw, blockIdx.x - nx);
    else
        bias_block(b, static_cast<int>(blockIdx.x - nx - nw));
}

constexpr int SUM_COLS = 256, SUM_ROWS = 4 * NWAVE;  // columns of a block of k_dpre, rows that it has in flight

struct Dpre {
    Mat grad, pre;        // pre: data NULL without an activation
    int M, N, act, rows;  // rows of a block
    float *dpre;          // [M, pitch]; NULL: not wanted
    int pitch;
    float *sums;          // [blocks of rows, N4]; NULL: not wanted
    int N4;
};

// dpre of a block's rows and columns, and their sums over the rows: 4 waves take every 4th row, 4 columns a lane.
template <bool GF32, bool PF32>
__global__ __launch_bounds__(NT) void k_dpre(Dpre d)
{
    __shared__ float part[NWAVE][SUM_COLS];
    const int wave = threadIdx.x >> 6, c = static_cast<int>(blockIdx.x) * SUM_COLS + 4 * (threadIdx.x & 63);
    const int m0 = static_cast<int>(blockIdx.y) * d.rows, m1 = m0 + d.rows < d.M ? m0 + d.rows : d.M, n = d.N - c;
    const bool act = d.pre.data;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
        for (int m = m0 + wave; m < m1; m += SUM_ROWS) {
            float g[4][4], p[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at = m + u * NWAVE < m1 ? m + u * NWAVE : m1 - 1;
                get4(d.grad.data, GF32, d.grad.row(at) + c, n, g[u]);
                if (act)
                    get4(d.pre.data, PF32, d.pre.row(at) + c, n, p[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (m + u * NWAVE >= m1)
                    break;
                if (act)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        g[u][e] *= slope_of(p[u][e], d.act);
                if (d.dpre)
                    *reinterpret_cast<f32x4 *>(d.dpre + static_cast<int64_t>(m + u * NWAVE) * d.pitch + c) =
                        f32x4{g[u][0], g[u][1], g[u][2], g[u][3]};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] += g[u][e];
            }
        }
    }
    if (!d.sums)
        return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        part[wave][4 * (threadIdx.x & 63) + e] = sum[e];
    __syncthreads();
    const int col = static_cast<int>(blockIdx.x) * SUM_COLS + static_cast<int>(threadIdx.x);
    if (col < d.N)
        d.sums[static_cast<int64_t>(blockIdx.y) * d.N4 + col] =
            (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}

}  // namespace DH_NS

namespace dhlinear {

using namespace dhl;

namespace {

int up(int64_t n, int64_t d) { return static_cast<int>((n + d - 1) / d); }
size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

struct Cut {
    int shape, ti, tj, splits, pitch;
    bool joined;   // the sums go out through k_gemm_join
    size_t bytes;  // of the parts
};

// Tiles.  bf: both operands are bfloat16; few: there are tiles for up to 16 rows (forward: 16 float32 rows of 256 by
// 151936 x 256 bfloat16 weights 21 us, in tiles of 64 rows 31; backward, 25 us either way).
// HUGE: where both sides of the result fill more than one tile of 128, else most of the tile is padding.  bfloat16, in tiles
// of 64, 128 and 256 squared: rows of 4096 by 151936 weights, 17 rows 221, 245, 390 us, 64 rows 266, 260, 396, 128 rows
// 361, 286, 404, 129 rows -, 424, 395, 512 rows 1168, 791, 677; gradient of w from 512 rows, 151936 x 16 53, 52, 85, x 128
// 83, 55, 84, x 192 114, 90, 84, x 256 145, 91, 84.  The shortest sum is 512: below, the two lie closer (gradient of w,
// 151936 x 256 from 496, 384, 256 rows: tiles of 128 94, 76, 56, of 256 87, 71, 54; 512 x 384 -> 151936 with a float32
// residual 182 and 181, x 256 152 and 157).
// LARGE: from 2048 steps of 64 on, about where they cross: in tiles of 64 and 128, bfloat16, 2048 x 512 -> 2048 13.4 and 12.7
// us, 1024 x 2048 -> 1024 18.5 and 21.8, 2048 x 1024 -> 1024 13.4 and 18.3 (float32 36 and 42); below it, 512 x 4096 -> 512
// 15.7 and 18.5, 1024 x 1024 -> 1024 9.7 and 18.
Cut cut_of(int64_t I, int64_t J, int64_t K, bool bf, bool few, int act = DOMINO_NO_ACT)
{
    static const int BI[] = {128, 64, 64, 256}, BJ[] = {128, 64, 16, 256};
    Cut c;
    const auto tiles = [&](int shape) { return static_cast<int64_t>(up(I, BI[shape])) * up(J, BJ[shape]); };
    const int64_t steps = up(K, 64);
    c.shape = few && J <= 16 ? FEW
              : bf && I > 128 && J > 128 && tiles(HUGE) >= 256 && K >= 512 ? HUGE
              : I >= 128 && J >= 128 && tiles(LARGE) * steps >= 2048 ? LARGE : MEDIUM;
    c.ti = up(I, BI[c.shape]), c.tj = up(J, BJ[c.shape]);
    // Few tiles share out their sums.  A part costs the join as I J does and saves steps as K does: 50 sqrt(K / (I J))
    // parts are best, or what makes one or two blocks a compute unit of them (512 x 256 results over K = 5120: 1, 4, 10,
    // 20, 40 parts 68, 22, 13.3, 15.6, 21 us; over 151936: 32, 64, 96 parts 82, 77, 84 us).  A short sum is not worth
    // the second launch (256 x 1024 over 1024, bfloat16: 9.2 us in one part, 13.3 in four; 203 x 1091 over 331, float32:
    // 20.9 and 15.2 us).
    const int64_t count = tiles(c.shape);
    int64_t n = count ? static_cast<int64_t>(std::ceil(50 * std::sqrt(static_cast<double>(K) /
                                                                     (static_cast<double>(I) * J)))) : 1;
    for (int blocks = 256; count && blocks <= 512; blocks += 256)
        if (10 * n >= 7 * (blocks / count))
            n = blocks == 512 || 10 * n < 7 * (512 / count) ? blocks / count : n;
    n = n < K / 64 ? n : K / 64;
    c.splits = n < 1 || K < (bf ? 1536 : 320) || c.shape == HUGE ? 1 : static_cast<int>(n);
    c.pitch = up(I, 4) * 4;
    c.joined = c.splits > 1 || act == DOMINO_GELU;
    c.bytes = c.joined ? static_cast<size_t>(c.splits) * J * c.pitch * sizeof(float) : 0;
    return c;
}

Gemm gemm_of(const Cut &c, const Mat &a, const Mat &b, int64_t I, int64_t J, int64_t K, void *ws)
{
    Gemm g = {};
    g.a = a, g.b = b;
    g.I = static_cast<int>(I), g.J = static_cast<int>(J), g.K = static_cast<int>(K);
    g.ti = c.ti, g.tj = c.tj, g.splits = c.splits;
    g.i_inner = c.ti <= c.tj;
    g.partial = c.joined ? static_cast<float *>(ws) : nullptr;
    g.pitch = c.pitch;
    return g;
}

void stream_of(Gemm &g)
{
    // large results, and a residual with them, go past the dies' caches: float32 logits of 151936 with a residual, 512
    // rows: 150 us, through the caches 166; 16 rows: 20.8 and 24.6 us
    const int64_t size = (g.e.out.f32 ? 4 : 2) + (g.e.residual.data ? g.e.residual.f32 ? 4 : 2 : 0);
    g.e.stream = size * g.I * g.J > 4 << 20;
}

unsigned join_blocks(const Gemm &g) { return up(static_cast<int64_t>(g.J) * (g.pitch / 4), NT); }
Divisor join_divisor(const Gemm &g) { return divisor(static_cast<uint32_t>(g.pitch / 4)); }

template <typename F>
hipError_t run(const Gemm &g, const Cut &c, F product, hipStream_t st)
{
    const hipError_t e = product(g, c.shape, st);
    if (e != hipSuccess || !c.joined)
        return e;
    hipLaunchKernelGGL(k_gemm_join, dim3(join_blocks(g)), dim3(NT), 0, st, g, join_divisor(g));
    return hipGetLastError();
}

int64_t rows(const domino_rows &m) { return static_cast<int64_t>(m.B) * m.R; }
bool bfloat(const domino_rows &a, const domino_rows &b) { return a.dtype == DOMINO_BF16 && b.dtype == DOMINO_BF16; }

}  // namespace

size_t workspace_bytes(const Forward &f) { return cut_of(f.weight->R, rows(*f.x), f.x->V, bfloat(*f.x, *f.weight), true, f.act).bytes; }

hipError_t forward(const Forward &f, void *ws, hipStream_t st)
{
    const int64_t M = rows(*f.x), N = f.weight->R, K = f.x->V;
    const Cut c = cut_of(N, M, K, bfloat(*f.x, *f.weight), true, f.act);
    Gemm g = gemm_of(c, mat_of(*f.weight), mat_of(*f.x), N, M, K, ws);
    g.e.out = mat_of(*f.y);
    if (f.pre)
        g.e.pre = mat_of(*f.pre);
    if (f.residual)
        g.e.residual = mat_of(*f.residual);
    if (f.bias)
        g.e.bias = f.bias->data, g.e.bias_f32 = f.bias->dtype == DOMINO_F32;
    g.e.act = f.act;
    stream_of(g);
    return run(g, c, product_y, st);
}

namespace {

struct Layout {
    Cut x, w;
    bool pair;  // both products in one launch
    int pitch, sum_rows, sum_blocks, N4;
    size_t dpre, sums, parts_x, parts_w, bytes;
};

Layout layout_of(const Backward &b)
{
    Layout l = {};
    const int64_t M = rows(*b.grad), N = b.weight->R, K = b.x->V;
    const bool act = b.act != DOMINO_NO_ACT;
    size_t at = 0;
    l.pitch = l.N4 = up(N, 4) * 4;
    l.dpre = at;
    if (act)
        at += static_cast<size_t>(M) * l.pitch * sizeof(float);
    // about 512 blocks: 64 to 256 of rows, of 4 rows or of multiples of 16 (331 rows of 203, gelu: 4 rows a block 4.7 us, 16
    // 7.7; 16384 rows of 256, silu and bias, a call: 256 blocks of rows 28 us, 64 83)
    const int most = std::min(256, std::max(64, up(512, up(N, SUM_COLS))));
    l.sum_rows = M > most * NWAVE ? up(M, most * SUM_ROWS) * SUM_ROWS : NWAVE;
    l.sum_blocks = up(M, l.sum_rows);
    l.sums = at;
    if (b.grad_bias)
        at += round16(static_cast<size_t>(l.sum_blocks) * l.N4 * sizeof(float));
    if (b.grad_x && M)
        l.x = cut_of(K, M, N, !act && bfloat(*b.grad, *b.weight), false);
    if (b.grad_weight)
        l.w = cut_of(K, N, M, !act && bfloat(*b.grad, *b.x), false);
    // (tiles of 64 x 64 have little to do; 331 x 1091 x 203, float32: 40 us a call in six launches, 26 in three)
    l.pair = b.grad_x && M && b.grad_weight && l.x.shape == MEDIUM && l.w.shape == MEDIUM;
    l.parts_x = l.parts_w = at;
    if (l.pair)
        l.parts_w += l.x.bytes;
    l.bytes = l.pair ? l.parts_w + l.w.bytes : at + (l.x.bytes > l.w.bytes ? l.x.bytes : l.w.bytes);
    return l;
}

}  // namespace

size_t workspace_bytes(const Backward &b) { return layout_of(b).bytes; }

hipError_t backward(const Backward &b, void *ws, hipStream_t st)
{
    const Layout l = layout_of(b);
    const int64_t M = rows(*b.grad), N = b.weight->R, K = b.x->V;
    char *base = static_cast<char *>(ws);
    Mat grad = mat_of(*b.grad);
    hipError_t e = hipSuccess;
    const bool act = b.act != DOMINO_NO_ACT;
    if (M && (act || b.grad_bias)) {
        Dpre d = {};
        d.grad = grad;
        if (act) {
            d.pre = mat_of(*b.pre);
            d.dpre = b.grad_x || b.grad_weight ? reinterpret_cast<float *>(base + l.dpre) : nullptr;
        }
        d.M = static_cast<int>(M), d.N = static_cast<int>(N), d.act = b.act, d.rows = l.sum_rows;
        d.pitch = l.pitch, d.N4 = l.N4;
        d.sums = b.grad_bias ? reinterpret_cast<float *>(base + l.sums) : nullptr;
        const bool pf32 = !act || d.pre.f32;
        const auto kernel = grad.f32 ? (pf32 ? k_dpre<true, true> : k_dpre<true, false>)
                                     : (pf32 ? k_dpre<false, true> : k_dpre<false, false>);
        hipLaunchKernelGGL(kernel, dim3(up(N, SUM_COLS), l.sum_blocks), dim3(NT), 0, st, d);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    if (act) {
        grad = Mat{};
        grad.data = base + l.dpre;
        grad.rs = l.pitch;
        grad.flat = grad.f32 = true;
        grad.near = grad.rs < (1 << 21);
    }
    Bias bias = {};
    if (b.grad_bias)
        bias = Bias{reinterpret_cast<float *>(base + l.sums), l.sum_blocks, static_cast<int>(N), l.N4,
                    mat_of(*b.grad_bias), b.accumulate};
    const unsigned bias_blocks = b.grad_bias ? up(N, 64) : 0;
    Gemm x = {}, w = {};
    if (b.grad_x && M) {
        x = gemm_of(l.x, mat_of(*b.weight), grad, K, M, N, base + l.parts_x);
        x.e.out = mat_of(*b.grad_x);
        stream_of(x);
    }
    if (b.grad_weight) {
        w = gemm_of(l.w, mat_of(*b.x), grad, K, N, M, base + l.parts_w);
        w.e.out = mat_of(*b.grad_weight);
        if (b.accumulate)
            w.e.residual = w.e.out;
        stream_of(w);
    }
    if (l.pair) {
        if ((e = product_pair(x, w, st)) != hipSuccess)
            return e;
    } else {
        if (b.grad_x && M && (e = run(x, l.x, product_dx, st)) != hipSuccess)
            return e;
        if (b.grad_weight && (e = run(w, l.w, product_dw, st)) != hipSuccess)
            return e;
    }
    const unsigned nx = l.pair && l.x.joined ? join_blocks(x) : 0, nw = l.pair && l.w.joined ? join_blocks(w) : 0;
    if (nx + nw + bias_blocks) {
        hipLaunchKernelGGL(k_join, dim3(nx + nw + bias_blocks), dim3(NT), 0, st, x, nx ? join_divisor(x) : Divisor{}, nx,
                           w, nw ? join_divisor(w) : Divisor{}, nw, bias);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace dhlinear
