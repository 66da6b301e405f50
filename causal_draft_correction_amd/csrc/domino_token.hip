// Log-probabilities of given tokens and the entropies of their rows, and the gradient of both.
//
// With p = softmax(z / tau), w the row's token, H = -sum p log p:
//     logprob = log p_w                dlogprob/dz_v = (1[v = w] - p_v) / tau
//     entropy = H                      dH/dz_v = -p_v (log p_v + H) / tau
// dh_score.h has the sums.  The forward pass reads a row once, one block per chunk with its values in registers
// (k_token_part), and joins the chunks in 64 bits (k_token_final); the backward pass reads it once and writes it once
// (k_token_grad): an element is e (a + b y) with y = log2 of e = p_v S and a, b the same for a row.  The token's own
// element is written again once the block's other stores are done, from 1 - p as the forward pass has it.  Rows that one
// block can hold go through one launch (k_token_row).
//
// Measured on one MI355X.  512 bfloat16 rows of 151936 (156 MB): forward 34.3 + 4.9 us, 4.6 TB/s: 439 vector instructions a
// wave, with two sums for each exponential, are as much a bound as the bytes; backward 44.6 us, 7.0 TB/s read and
// written, part of it from the last-level cache, where the forward pass left the rows.  768 float32 rows of 50021, half of
// them left out: 17.7 + 4.9 + 40.6 us; the gradient's zeros for rows left out are half its stores.
#define DH_NT 256
#define DH_NS dhk
#include "dh_score.h"
#include "dh_token.h"

namespace DH_NS {

static_assert(SCORE_STATS == dhtoken::STATS, "");

// The block's part, in every thread.
template <typename T, int NV, int NTB>
__device__ inline ScorePart chunk_score(typename Vec<T>::raw (&x)[NV], const T *row, int V, int c, int cvec,
                                        const Scale &sc, float *red_m, double (*red)[2])
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    float mine = NEG_INF;
#pragma unroll
    for (int u = 0; u < NV; ++u)
        mine = Vec<T>::max_with(x[u], mine);
    const float wm = wave_max(mine);
    if (lane == 0)
        red_m[wave] = wm;
    __syncthreads();
    float m = red_m[0];
#pragma unroll
    for (int w = 1; w < NTB / 64; ++w)
        m = fmaxf(m, red_m[w]);
    const Expo ex(m > NEG_INF ? m : 0.f, sc);
    bool odd;
    return block_score<T, NV, NTB>(x, row, V, c, cvec, mine, m, red_m, red, ex, sc, odd);
}

// The chunk's elements of the gradient; not live: zeros.
struct Coef {
    float a, b;  // e (a + b y)
    float token;
};
__device__ inline Coef coef_of(const float (&st)[SCORE_STATS], const Expo &ex, const Scale &sc, float g_logprob,
                               float g_entropy, float inv_tau)
{
    Coef c;
    const float k = st[1] * static_cast<float>(ex.fix(sc)) * inv_tau;
    c.b = -g_entropy * static_cast<float>(LN2) * k;
    c.a = -fmaf(g_entropy, st[2], g_logprob) * k - c.b * static_cast<float>(ex.off(sc));
    c.token = (g_logprob * st[5] - g_entropy * st[6]) * inv_tau;
    return c;
}

template <typename T, int NV>
__device__ inline void chunk_grad(typename Vec<T>::raw (&x)[NV], bool live, const Expo &ex, const Scale &sc, const Coef &c)
{
    if (!live) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            x[u] = typename Vec<T>::raw{0, 0, 0, 0};
    } else if (c.b == 0.f) {
        if (ex.small) {
#pragma unroll
            for (int u = 0; u < NV; ++u)
                Vec<T>::map(x[u], [&](float z) { return c.a * ex.at<true>(z, sc); });
        } else {
#pragma unroll
            for (int u = 0; u < NV; ++u)
                Vec<T>::map(x[u], [&](float z) { return c.a * ex.at<false>(z, sc); });
        }
    } else {
        const auto one = [&](float y) {
            return __builtin_amdgcn_exp2f(y) * fmaf(c.b, fmaxf(y, -1000.f), c.a);
        };
        if (ex.small) {
#pragma unroll
            for (int u = 0; u < NV; ++u)
                Vec<T>::map(x[u], [&](float z) { return one(ex.exponent<true>(z, sc)); });
        } else {
#pragma unroll
            for (int u = 0; u < NV; ++u)
                Vec<T>::map(x[u], [&](float z) { return one(ex.exponent<false>(z, sc)); });
        }
    }
}

template <typename T, int NV>
__global__ __launch_bounds__(NT) void k_token_part(Rows rows, Score score, Split sp, bool keep, Scale sc, ScorePart *parts)
{
    __shared__ float red_m[NWAVE];
    __shared__ double red[NWAVE][2];
    const int i_row = static_cast<int>(sp.by.quotient(blockIdx.x)), c = static_cast<int>(blockIdx.x) - i_row * sp.nch;
    const Place place = rows.place(i_row);
    if (!score_counts(rows, score, place))
        return;
    typename Vec<T>::raw x[NV];
    const T *z = row_at<T>(rows, place);
    if (keep)
        load_chunk<T, NV, NT, true>(x, z, rows.V, c, sp.cvec);
    else
        load_chunk<T, NV>(x, z, rows.V, c, sp.cvec);
    const ScorePart part = chunk_score<T, NV, NT>(x, z, rows.V, c, sp.cvec, sc, red_m, red);
    if (threadIdx.x == 0)
        parts[static_cast<int64_t>(place.row) * sp.nch + c] = part;
}

// One row a wave.
template <typename T>
__global__ __launch_bounds__(NT) void k_token_final(Rows rows, Score score, int n_all, int nch, double inv_tau,
                                                    const ScorePart *parts)
{
    const int i = blockIdx.x * NWAVE + static_cast<int>(threadIdx.x >> 6);
    if (i >= n_all)
        return;
    const Place place = rows.place(i);
    const int lane = threadIdx.x & 63, row = place.row;
    if (!score_counts(rows, score, place)) {
        if (lane == 0)
            no_score(score, row);
        return;
    }
    const ScorePart *mine = parts + static_cast<int64_t>(row) * nch;
    const ScorePart first = first_part(mine, nch);
    const float z = Vec<T>::one(row_at<T>(rows, place) + score.tokens[row]);
    const ScorePart all = join_parts(first, mine, nch, inv_tau);
    const double log_s = log1p(all.s);
    if (lane == 0)
        put_score(score, row, z, all, log_s, inv_tau,
                  score.stats ? score.stats + static_cast<int64_t>(row) * SCORE_STATS : nullptr);
}

__device__ inline float grad_at(const float *g, int row) { return g ? g[row] : 0.f; }

template <typename T, int NV>
__global__ __launch_bounds__(NT) void k_token_grad(Rows rows, Score score, Split sp, const float *g_logprob,
                                                   const float *g_entropy, float inv_tau, Scale sc, Rows grad)
{
    const int i_row = static_cast<int>(sp.by.quotient(blockIdx.x)), c = static_cast<int>(blockIdx.x) - i_row * sp.nch;
    const Place place = rows.place(i_row);
    T *out = const_cast<T *>(row_at<T>(grad, place));
    const int v0 = chunk_begin<T>(c, sp.cvec, rows.V), v1 = chunk_begin<T>(c + 1, sp.cvec, rows.V);
    typename Vec<T>::raw x[NV];
    const bool counts = score_counts(rows, score, place);
    float st[SCORE_STATS] = {};
    if (counts) {
        load_chunk<T, NV>(x, row_at<T>(rows, place), rows.V, c, sp.cvec);
#pragma unroll
        for (int i = 0; i < SCORE_STATS; ++i)
            st[i] = score.stats[static_cast<int64_t>(place.row) * SCORE_STATS + i];
    }
    const bool live = counts && st[3] != 0.f;
    const Expo ex(st[0], sc);
    const Coef coef = coef_of(st, ex, sc, grad_at(g_logprob, place.row), grad_at(g_entropy, place.row), inv_tau);
    chunk_grad<T, NV>(x, live, ex, sc, coef);
    store_chunk<T, NV>(x, out, v0, v1);
    if (!live)
        return;
    const int token = score.tokens[place.row];
    if (token < v0 || token >= v1)
        return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the block's stores are done
    __syncthreads();
    if (threadIdx.x == 0)
        Vec<T>::put(out + token, coef.token);
}

// A row of at most NV vectors a thread, by one block: its results, and with GRAD its gradient (the row is read once).
template <typename T, int NTB, int NV, bool GRAD>
__global__ __launch_bounds__(NTB) void k_token_row(Rows rows, Score score, double inv_tau, Scale sc, const float *g_logprob,
                                                  const float *g_entropy, Rows grad)
{
    typedef Vec<T> VT;
    __shared__ float red_m[NTB / 64];
    __shared__ double red[NTB / 64][2];
    __shared__ float s_stat[SCORE_STATS];
    const Place place = rows.place(blockIdx.x);
    const int row = place.row;
    const bool counts = score_counts(rows, score, place);
    typename VT::raw x[NV];
    if (counts) {
        const T *z = row_at<T>(rows, place);
        load_chunk<T, NV, NTB>(x, z, rows.V, 0, NV * NTB);
        const ScorePart part = chunk_score<T, NV, NTB>(x, z, rows.V, 0, NV * NTB, sc, red_m, red);
        if (threadIdx.x == 0)
            put_score(score, row, VT::one(z + score.tokens[row]), part, log1p(part.s), inv_tau,
                      GRAD ? s_stat
                           : score.stats ? score.stats + static_cast<int64_t>(row) * SCORE_STATS : nullptr);
    } else if (threadIdx.x == 0) {
        no_score(score, row);
        if constexpr (GRAD)
            for (int i = 0; i < SCORE_STATS; ++i)
                s_stat[i] = 0.f;
    }
    if constexpr (GRAD) {
        __syncthreads();
        T *out = const_cast<T *>(row_at<T>(grad, place));
        float st[SCORE_STATS];
#pragma unroll
        for (int i = 0; i < SCORE_STATS; ++i)
            st[i] = s_stat[i];
        const bool live = st[3] != 0.f;
        const Expo ex(st[0], sc);
        const Coef coef = coef_of(st, ex, sc, grad_at(g_logprob, row), grad_at(g_entropy, row),
                                  static_cast<float>(inv_tau));
        forget(x);
        chunk_grad<T, NV>(x, live, ex, sc, coef);
        store_chunk<T, NV, NTB>(x, out, 0, rows.V);
        if (live) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the block's stores are done
            __syncthreads();
            if (threadIdx.x == 0)
                VT::put(out + score.tokens[row], coef.token);
        }
    }
}

}  // namespace DH_NS

namespace dhtoken {

using namespace dhk;

namespace {

constexpr int TARGET_BLOCKS = 1024;
// Vectors a thread takes at most, forward and backward.  With 8 the forward pass alone of 512 bfloat16 rows of 151936 is
// 2 us shorter (36 of 38), but its gradient then 3 us longer (47.7 of 44.6: it finds less of the rows in the caches); float32,
// 52 and 50 us forward, 104 either way backward.
constexpr int NV = 4;

int vectors(const domino_logits &lg)
{
    const int per = lg.dtype == DOMINO_F32 ? 4 : 8;
    return static_cast<int>((static_cast<int64_t>(lg.V) + per - 1) / per);
}

// Rows that one block takes whole, by the same sizes as those of a distillation, whose passes are alike: up to 8 vectors
// for each of 1024 threads where a gradient follows or every row has a compute unit for itself, else of 512.
bool whole_rows(const domino_logits &lg, bool grad)
{
    const int nvec = vectors(lg);
    return nvec <= 512 * 8 || (nvec <= 1024 * 8 && (grad || static_cast<int64_t>(lg.B) * lg.R <= 256));
}

Split split_of(const domino_logits &lg)
{
    const int64_t rows = static_cast<int64_t>(lg.B) * lg.R;
    const int nvec = vectors(lg);
    const int least = static_cast<int>((static_cast<int64_t>(nvec) + NT * NV - 1) / (NT * NV));
    int64_t n = rows ? (TARGET_BLOCKS + rows - 1) / rows : 1;
    n = n < nvec / NT ? n : nvec / NT;
    n = n > least ? n : least;
    return split(nvec, n);
}

template <typename F>
void by_type(int dtype, F f)
{
    if (dtype == DOMINO_F32)
        f(float{});
    else
        f(bf16s{});
}

unsigned rows_of_call(const domino_logits &lg) { return static_cast<unsigned>(lg.B) * static_cast<unsigned>(lg.R); }

size_t parts_bytes(const domino_logits &lg)
{
    const size_t n = static_cast<size_t>(lg.B) * lg.R * split_of(lg).nch * sizeof(ScorePart);
    return (n + 15) & ~static_cast<size_t>(15);
}

Score score_of(const Scores &s, float *stats) { return Score{s.tokens, s.logprob, s.entropy, stats}; }

template <bool GRAD>
hipError_t by_rows(const domino_logits &lg, const Scores &s, double tau, const int32_t *n_rows, const float *g_logprob,
                   const float *g_entropy, const domino_logits *grad, hipStream_t st)
{
    const int nvec = vectors(lg);
    const Rows rows = rows_of(lg, n_rows, n_rows != nullptr), out = grad ? rows_of(*grad, nullptr, false) : Rows{};
    const dim3 grid(rows_of_call(lg));
    const Score score = score_of(s, s.stats);
    const Scale sc = scale_of(tau);
    by_type(lg.dtype, [&](auto type) {
        typedef decltype(type) T;
        if (nvec <= 256 * 2)
            hipLaunchKernelGGL((k_token_row<T, 256, 2, GRAD>), grid, dim3(256), 0, st, rows, score, 1.0 / tau, sc,
                               g_logprob, g_entropy, out);
        else if (nvec <= 256 * 8)
            hipLaunchKernelGGL((k_token_row<T, 256, 8, GRAD>), grid, dim3(256), 0, st, rows, score, 1.0 / tau, sc,
                               g_logprob, g_entropy, out);
        else if (nvec <= 512 * 8)
            hipLaunchKernelGGL((k_token_row<T, 512, 8, GRAD>), grid, dim3(512), 0, st, rows, score, 1.0 / tau, sc,
                               g_logprob, g_entropy, out);
        else
            hipLaunchKernelGGL((k_token_row<T, 1024, 8, GRAD>), grid, dim3(1024), 0, st, rows, score, 1.0 / tau, sc,
                               g_logprob, g_entropy, out);
    });
    return hipGetLastError();
}

// keep: the logits may stay in the caches, for a gradient that follows.
hipError_t in_parts(const domino_logits &lg, const Scores &s, float *stats, double tau, const int32_t *n_rows, void *ws,
                    bool keep, hipStream_t st)
{
    const Rows rows = rows_of(lg, n_rows, n_rows != nullptr);
    const Split sp = split_of(lg);
    const unsigned n = rows_of_call(lg);
    const Score score = score_of(s, stats);
    const Scale sc = scale_of(tau);
    ScorePart *parts = static_cast<ScorePart *>(ws);
    by_type(lg.dtype, [&](auto type) {
        typedef decltype(type) T;
        const dim3 grid(n * sp.nch);
        if (sp.nv <= 2)
            hipLaunchKernelGGL((k_token_part<T, 2>), grid, dim3(NT), 0, st, rows, score, sp, keep, sc, parts);
        else
            hipLaunchKernelGGL((k_token_part<T, NV>), grid, dim3(NT), 0, st, rows, score, sp, keep, sc, parts);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    by_type(lg.dtype, [&](auto type) {
        hipLaunchKernelGGL((k_token_final<decltype(type)>), dim3((n + NWAVE - 1) / NWAVE), dim3(NT), 0, st, rows, score,
                           static_cast<int>(n), sp.nch, 1.0 / tau, parts);
    });
    return hipGetLastError();
}

// Sizes up to which the forward pass leaves the logits in the caches: where its gradient follows, and where one may.
constexpr double KEEP_FOR_GRAD = 512e6, KEEP_FOR_STATS = 256e6;

double bytes_of(const domino_logits &lg)
{
    return static_cast<double>(lg.B) * lg.R * lg.V * (lg.dtype == DOMINO_F32 ? 4 : 2);
}

}  // namespace

size_t workspace_bytes(const domino_logits &lg)
{
    if (whole_rows(lg, false))
        return 0;
    return parts_bytes(lg) + static_cast<size_t>(lg.B) * lg.R * SCORE_STATS * sizeof(float);
}

hipError_t forward(const domino_logits &lg, const Scores &s, double tau, const int32_t *n_rows, void *ws, hipStream_t st)
{
    if (whole_rows(lg, false))
        return by_rows<false>(lg, s, tau, n_rows, nullptr, nullptr, nullptr, st);
    return in_parts(lg, s, s.stats, tau, n_rows, ws, s.stats && bytes_of(lg) <= KEEP_FOR_STATS, st);
}

hipError_t backward(const domino_logits &lg, const int32_t *tokens, const float *stats, const float *grad_logprob,
                    const float *grad_entropy, double tau, const int32_t *n_rows, const domino_logits &grad,
                    hipStream_t st)
{
    const Rows rows = rows_of(lg, n_rows, n_rows != nullptr), out = rows_of(grad, nullptr, false);
    const Split sp = split_of(lg);
    const dim3 grid(rows_of_call(lg) * sp.nch);
    const Score score = {tokens, nullptr, nullptr, const_cast<float *>(stats)};
    const float inv_tau = static_cast<float>(1.0 / tau);
    const Scale sc = scale_of(tau);
    by_type(lg.dtype, [&](auto type) {
        typedef decltype(type) T;
        if (sp.nv <= 2)
            hipLaunchKernelGGL((k_token_grad<T, 2>), grid, dim3(NT), 0, st, rows, score, sp, grad_logprob, grad_entropy,
                               inv_tau, sc, out);
        else
            hipLaunchKernelGGL((k_token_grad<T, NV>), grid, dim3(NT), 0, st, rows, score, sp, grad_logprob,
                               grad_entropy, inv_tau, sc, out);
    });
    return hipGetLastError();
}

hipError_t both(const domino_logits &lg, const Scores &s, double tau, const int32_t *n_rows, void *ws,
                const float *grad_logprob, const float *grad_entropy, const domino_logits &grad, hipStream_t st)
{
    if (whole_rows(lg, true))
        return by_rows<true>(lg, s, tau, n_rows, grad_logprob, grad_entropy, &grad, st);
    float *stats = reinterpret_cast<float *>(static_cast<char *>(ws) + parts_bytes(lg));
    const hipError_t e = in_parts(lg, s, stats, tau, n_rows, ws, bytes_of(lg) <= KEEP_FOR_GRAD, st);
    return e == hipSuccess ? backward(lg, s.tokens, stats, grad_logprob, grad_entropy, tau, n_rows, grad, st) : e;
}

}  // namespace dhtoken
