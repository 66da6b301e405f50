// The largest logits of vocabulary rows, and one step of beam search over them.
//
// top: for each row z of [B, R, V] logits the k largest (largest first; ties to the lowest id, NaN above every
// number, -0 == +0) and lse = log sum_v exp(z_v / tau).  Both follow from one reading of the row, so the work
// is bound by HBM bandwidth for many rows and by latency for few.
//
// k_top_chunk: one block takes one chunk of a row into registers.  Each thread's maximum is a candidate; the
// ceil(k/4)-th largest of a wave's 64 maxima, the lowest of the four waves', is a bound that at least k elements
// of the chunk reach and (on rows in no particular order) about 1.5 k to 3 k do.  It is found by 32 ballots and no
// exchange.  The elements that reach it go to a list in LDS, and the place of each among the largest is the
// number of greater ones.
// k_top_merge joins the chunks' lists of a row the same way.
//
// beam: W beams' candidates score s_w + z_wv - lse_w.  Within a beam they are ordered by their logits, so the
// M best of all are among the M largest of each row; k_beam_merge ranks these by binary searches in the other
// beams' lists and writes state and history in the new order.
#define DH_NT 256
#define DH_NS dht
#include "dh_rows.h"
#include "dh_top.h"

namespace DH_NS {

constexpr int LIST = 2048;         // candidates of a chunk that the LDS list holds
constexpr int MERGE_LIST = 4096;   // candidates of a row's chunks
constexpr int MAX_TIES = 128;      // of them kept for elements equal to the bound (at least MAX_K)
constexpr int COUNT_MAX = 256;     // up to here places are counted, above the list is sorted
constexpr int MAX_BEAMS = dhtop::MAX_W, MAX_OUT = dhtop::MAX_K;
static_assert(MAX_TIES >= dhtop::MAX_K, "the ties alone may be the result");

// Rows that are not read: past n_rows; beams that are dead (score -inf), ended, or without a usable score.
struct Live {
    const float *scores;
    const uint8_t *finished;
};
__device__ inline bool row_live(const Rows &rows, const Live &lv, int row)
{
    const int b = row / rows.R, r = row % rows.R;
    if (lv.scores) {
        const float s = lv.scores[row];
        return s > NEG_INF && s < -NEG_INF && !(lv.finished && lv.finished[row]);
    }
    return rows.counts(b, r);
}

// Unsigned words in the order of finite and infinite floats, 0 below all of them.
__device__ inline uint32_t ord_f32(float f)
{
    const uint32_t u = __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ inline float unord_f32(uint32_t o)
{
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}
__device__ inline float key_value(uint64_t key) { return unord_f32(static_cast<uint32_t>(key >> 32)); }

// Largest t that at least n lanes reach (0 if fewer than n lanes hold more than 0).
__device__ inline uint32_t wave_nth(uint32_t v, int n)
{
    uint32_t t = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = t | (1u << bit);
        if (__popcll(__ballot(v >= c)) >= n)
            t = c;
    }
    return t;
}
__device__ inline uint64_t wave_nth(uint64_t v, int n)
{
    const uint32_t hi = wave_nth(static_cast<uint32_t>(v >> 32), n);
    const bool tie = static_cast<uint32_t>(v >> 32) == hi;
    const int above = __popcll(__ballot(static_cast<uint32_t>(v >> 32) > hi));
    const uint32_t lo = wave_nth(tie ? static_cast<uint32_t>(v) : 0u, n - above);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// Sorts list[0, n) in descending order (n <= LEN; list holds the next power of two).
__device__ inline void block_sort(uint64_t *list, int n)
{
    int len = 2;
    while (len < n)
        len <<= 1;
    for (int i = n + static_cast<int>(threadIdx.x); i < len; i += NT)
        list[i] = 0;
    for (int size = 2; size <= len; size <<= 1)
        for (int step = size >> 1; step; step >>= 1) {
            __syncthreads();
            for (int i = threadIdx.x; i < len / 2; i += NT) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const uint64_t x = list[a], y = list[b];
                if ((x < y) == ((a & size) == 0))
                    list[a] = y, list[b] = x;
            }
        }
    __syncthreads();
}

// Hands the k largest of list[0, n) to emit(place, key), largest first; places past n get key 0.
template <typename F>
__device__ inline void emit_largest(uint64_t *list, int n, int k, F emit)
{
    if (n > COUNT_MAX) {
        block_sort(list, n);
        for (int i = threadIdx.x; i < k; i += NT)
            emit(i, list[i]);
        return;
    }
    const int t = threadIdx.x;
    if (t < n) {
        const uint64_t key = list[t];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j)
            place += list[j] > key;
        if (place < k)
            emit(place, key);
    }
    for (int i = n + t; i < k; i += NT)
        emit(i, 0ull);
}

struct ChunkShared {
    uint64_t list[LIST];
    uint64_t best[NWAVE];
    float m[NWAVE], s[NWAVE];
    uint32_t t[NWAVE];
    int n, ties;
};

__device__ inline float block_max(float v, float *red)
{
    const int wave = threadIdx.x >> 6;
    v = wave_max(v);
    if ((threadIdx.x & 63) == 0)
        red[wave] = v;
    __syncthreads();
    float m = red[0];
#pragma unroll
    for (int w = 1; w < NWAVE; ++w)
        m = fmaxf(m, red[w]);
    return m;
}

// The k largest of row[v0, v1) by k passes, each for the largest key below the last: any values, NaN and
// infinities among them.  For rows with such values and for orders that overflow the list.
template <typename T, typename F>
__device__ inline void largest_by_rounds(const T *row, int v0, int v1, int k, ChunkShared &sh, F emit)
{
    uint64_t last = ~0ull;
    for (int i = 0; i < k; ++i) {
        uint64_t best = 0;
        for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += NT) {
            const uint64_t key = argmax_key(Vec<T>::one(row + v), static_cast<uint32_t>(v));
            if (key < last && key > best)
                best = key;
        }
        best = wave_max_u64(best);
        if ((threadIdx.x & 63) == 0)
            sh.best[threadIdx.x >> 6] = best;
        __syncthreads();
        best = sh.best[0];
#pragma unroll
        for (int w = 1; w < NWAVE; ++w)
            best = max_u64(best, sh.best[w]);
        __syncthreads();
        if (threadIdx.x == 0)
            emit(i, best);
        last = best;  // 0 once nothing is left
    }
}

// More elements than the list holds reach the bound t, most of them equal to it (masked rows: all the rest is
// -inf).  The greater ones go to the list, then the equal ones in the order of their ids until k are there.
// False: too many are greater.
template <typename T>
__device__ inline bool list_with_ties(const T *row, int v0, int v1, float t, int k, ChunkShared &sh)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
    if (threadIdx.x == 0)
        sh.n = 0;
    __syncthreads();
    for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += NT) {
        const float z = Vec<T>::one(row + v);
        if (z > t) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < LIST - MAX_TIES)
                sh.list[at] = argmax_key(z, static_cast<uint32_t>(v));
        }
    }
    __syncthreads();
    const int greater = sh.n;
    if (greater > LIST - MAX_TIES)
        return false;
    int have = 0;  // equal ones so far
    for (int base = v0; base < v1 && greater + have < k; base += NT) {
        const int v = base + static_cast<int>(threadIdx.x);
        const bool tie = v < v1 && Vec<T>::one(row + v) == t;
        const uint64_t mask = __ballot(tie);
        if (lane == 0)
            sh.t[wave] = __popcll(mask);
        __syncthreads();
        int before = have, all = have;
#pragma unroll
        for (int w = 0; w < NWAVE; ++w) {
            before += w < wave ? static_cast<int>(sh.t[w]) : 0;
            all += static_cast<int>(sh.t[w]);
        }
        const int at = greater + before + __popcll(mask & ((1ull << lane) - 1));
        if (tie && at < k)
            sh.list[at] = argmax_key(t, static_cast<uint32_t>(v));
        have = all;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        sh.n = greater + have < k ? greater + have : (greater > k ? greater : k);
    __syncthreads();
    return true;
}

// What one block leaves of its chunk: keys and part, or (a row of one chunk) the results.
struct TopOut {
    uint64_t *keys;    // [rows, nch, k]
    Part *parts;       // [rows, nch]
    int32_t *ids;      // [rows, k]; NULL where keys and parts are wanted
    float *values, *lse;
};

__device__ inline void put_result(const TopOut &o, int row, int k, int place, uint64_t key)
{
    o.ids[static_cast<int64_t>(row) * k + place] = static_cast<int32_t>(key_index(key));
    o.values[static_cast<int64_t>(row) * k + place] = key_value(key);
}

template <typename T, int NV>
__global__ __launch_bounds__(NT) void k_top_chunk(Rows rows, Live live, int k, int nch, int cvec, Scale sc,
                                                  double inv_tau, TopOut out)
{
    typedef Vec<T> VT;
    __shared__ ChunkShared sh;
    const int row = blockIdx.x / nch, c = blockIdx.x % nch, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const bool direct = nch == 1 && out.ids;
    if (!row_live(rows, live, row)) {
        if (direct) {
            for (int i = threadIdx.x; i < k; i += NT) {
                out.ids[static_cast<int64_t>(row) * k + i] = -1;
                out.values[static_cast<int64_t>(row) * k + i] = NEG_INF;
            }
            if (threadIdx.x == 0)
                out.lse[row] = NEG_INF;
        }
        return;
    }
    const T *z = row_at<T>(rows, row / rows.R, row % rows.R);
    const int v0 = chunk_begin<T>(c, cvec, rows.V), v1 = chunk_begin<T>(c + 1, cvec, rows.V);
    typename VT::raw x[NV];
    load_chunk<T, NV>(x, z, rows.V, c, cvec);
    if (threadIdx.x == 0)
        sh.n = 0;

    float tm = NEG_INF;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < VT::N; ++e)
            tm = fmaxf(tm, VT::get(x[u], e));
    // the bound: a lane without an element counts as below everything
    const bool any = v0 + static_cast<int>(threadIdx.x) * VT::N < v1;
    const uint32_t t_wave = wave_nth(any ? ord_f32(tm) : 0u, (k + NWAVE - 1) / NWAVE);
    if (lane == 0)
        sh.t[wave] = t_wave;
    const float m = block_max(tm, sh.m);
    uint32_t t_ord = sh.t[0];
#pragma unroll
    for (int w = 1; w < NWAVE; ++w)
        t_ord = t_ord < sh.t[w] ? t_ord : sh.t[w];
    const float t = t_ord ? unord_f32(t_ord) : NEG_INF;

    const float ref = m > NEG_INF ? m : 0.f;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < VT::N; ++e) {
            const float f = VT::get(x[u], e);
            s += exp_scaled(f - ref, sc);
            if (f >= t) {
                const int v = v0 + (u * NT + static_cast<int>(threadIdx.x)) * VT::N + e;
                if (v < v1) {
                    const int at = atomicAdd(&sh.n, 1);
                    if (at < LIST)
                        sh.list[at] = argmax_key(f, static_cast<uint32_t>(v));
                }
            }
        }
    s = wave_sum(s);
    if (lane == 0)
        sh.s[wave] = s;
    __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < NWAVE; ++w)
        total += static_cast<double>(sh.s[w]);
    const int64_t slot = static_cast<int64_t>(row) * nch + c;
    auto emit = [&](int place, uint64_t key) {
        if (direct)
            put_result(out, row, k, place, key);
        else
            out.keys[slot * k + place] = key;
    };

    Part part = {m, static_cast<float>(total)};
    const int n = sh.n;
    if (total != total) {
        // NaN or +inf among the elements (+inf alone makes the maximum +inf)
        bool nan = false;
        for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += NT) {
            const float f = VT::one(z + v);
            nan |= f != f;
        }
        nan = __syncthreads_or(nan);
        part = nan ? Part{__builtin_nanf(""), 1.f} : Part{-NEG_INF, 1.f};
        total = 1.0;
        largest_by_rounds(z, v0, v1, k, sh, emit);
    } else if (n <= LIST) {
        emit_largest(sh.list, n, k, emit);
    } else if (list_with_ties(z, v0, v1, t, k, sh)) {
        emit_largest(sh.list, sh.n, k, emit);
    } else {
        largest_by_rounds(z, v0, v1, k, sh, emit);
    }
    if (threadIdx.x == 0) {
        if (direct)
            out.lse[row] = part.m == NEG_INF ? NEG_INF : static_cast<float>(part.m * inv_tau + log(total));
        else
            out.parts[slot] = part;
    }
}

// The k largest of a row from its chunks' lists, and its log-sum-exp.
struct MergeShared {
    uint64_t list[MERGE_LIST];
    uint64_t t[NWAVE];
    int n;
};

__device__ inline int merge_list(const uint64_t *keys, int n, int k, MergeShared &sh)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    uint64_t best = 0;
    for (int i = threadIdx.x; i < n; i += NT)
        best = max_u64(best, keys[i]);
    const uint64_t t_wave = wave_nth(best, (k + NWAVE - 1) / NWAVE);
    if (lane == 0)
        sh.t[wave] = t_wave;
    if (threadIdx.x == 0)
        sh.n = 0;
    __syncthreads();
    uint64_t t = sh.t[0];
#pragma unroll
    for (int w = 1; w < NWAVE; ++w)
        t = t < sh.t[w] ? t : sh.t[w];
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t key = keys[i];
        if (key >= t && key)
            sh.list[atomicAdd(&sh.n, 1)] = key;
    }
    __syncthreads();
    return sh.n;
}

__global__ __launch_bounds__(NT) void k_top_merge(Rows rows, Live live, int k, int nch, double inv_tau, TopOut out,
                                                  uint64_t *merged)
{
    __shared__ MergeShared sh;
    const int row = blockIdx.x;
    if (!row_live(rows, live, row)) {
        if (out.ids) {
            for (int i = threadIdx.x; i < k; i += NT) {
                out.ids[static_cast<int64_t>(row) * k + i] = -1;
                out.values[static_cast<int64_t>(row) * k + i] = NEG_INF;
            }
            if (threadIdx.x == 0)
                out.lse[row] = NEG_INF;
        }
        return;
    }
    const int64_t slot = static_cast<int64_t>(row) * nch;
    const int n = merge_list(out.keys + slot * k, nch * k, k, sh);
    emit_largest(sh.list, n, k, [&](int place, uint64_t key) {
        if (out.ids)
            put_result(out, row, k, place, key);
        else
            merged[static_cast<int64_t>(row) * k + place] = key;
    });
    if (out.ids && threadIdx.x < 64) {
        float m;
        double s;
        join_parts(out.parts + slot, nch, inv_tau, m, s);
        if (threadIdx.x == 0)
            out.lse[row] = m == NEG_INF ? NEG_INF : static_cast<float>(m * inv_tau + log(s));
    }
}

// Unsigned words in the order of doubles: NaN above +inf, -0 as +0.
__device__ inline uint64_t ord_f64(double d)
{
    const uint64_t u = d == 0.0 ? 0ull : __builtin_bit_cast(uint64_t, d);
    if (d != d)
        return ~0ull;
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

struct BeamArgs {
    int W, M, V, kc, nch, eos, T, step;
    int64_t state_bytes;
    const uint64_t *lists;   // [B * W, kc]: each live beam's largest logits, largest first
    const Part *parts;       // [B * W, nch]
    const float *scores;
    const uint8_t *finished;
    const char *state;
    const int32_t *history;
    float *o_scores;
    int32_t *o_parent, *o_token;
    uint8_t *o_finished;
    char *o_state;
    int32_t *o_history;
};

template <typename V>
__device__ inline void copy_rows(const char *src, char *dst, int64_t bytes, int M, const int *parent, int part,
                                 int nparts)
{
    const int64_t per = bytes / static_cast<int64_t>(sizeof(V)), all = per * M;
    for (int64_t i = static_cast<int64_t>(part) * NT + threadIdx.x; i < all; i += static_cast<int64_t>(nparts) * NT) {
        const int64_t j = i / per, e = i - j * per;
        reinterpret_cast<V *>(dst)[i] = reinterpret_cast<const V *>(src)[parent[j] * per + e];
    }
}

// One batch entry.  Its blocks (blockIdx.y) all rank the candidates and share the copying of the state; block 0
// writes the rest.  LDS: scores' words [W kc], tokens [W kc].
__global__ __launch_bounds__(NT) void k_beam_merge(BeamArgs a)
{
    extern __shared__ uint64_t dyn[];
    __shared__ double log_s[MAX_BEAMS];
    __shared__ float top[MAX_BEAMS];
    __shared__ double s_score[MAX_OUT];
    __shared__ int s_parent[MAX_OUT], s_token[MAX_OUT];
    const int b = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int n = a.W * a.kc;
    uint64_t *score = dyn;
    int *token = reinterpret_cast<int *>(dyn + n);
    for (int w = wave; w < a.W; w += NWAVE) {
        const int row = b * a.W + w;
        const float s = a.scores[row];
        if (s > NEG_INF && s < -NEG_INF && !(a.finished && a.finished[row])) {
            float m;
            double t;
            join_parts(a.parts + static_cast<int64_t>(row) * a.nch, a.nch, 1.0, m, t);
            if (lane == 0)
                top[w] = m, log_s[w] = log(t);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const int w = i / a.kc, j = i - w * a.kc, row = b * a.W + w;
        const double s = a.scores[row];
        double val;
        int tok = j;
        if (s == static_cast<double>(NEG_INF)) {           // dead
            val = static_cast<double>(NEG_INF);
        } else if (a.finished && a.finished[row]) {        // ended: the end token, then the others
            tok = j == 0 ? a.eos : (j - 1 < a.eos ? j - 1 : j);
            val = j == 0 ? s : static_cast<double>(NEG_INF);
        } else if (!(s < -static_cast<double>(NEG_INF)) || !(top[w] < -NEG_INF)) {
            val = __builtin_nan("");                       // no distribution
        } else {
            const uint64_t key = a.lists[static_cast<int64_t>(row) * a.kc + j];
            const double z = key_value(key);
            tok = static_cast<int>(key_index(key));
            // (z - max first: a row at the type's lowest value keeps its differences)
            val = z == static_cast<double>(NEG_INF) ? z : s + ((z - static_cast<double>(top[w])) - log_s[w]);
        }
        score[i] = ord_f64(val);
        token[i] = tok;
    }
    __syncthreads();
    // place of candidate (w, j): j, and the candidates of other beams that go before it (equal scores: the
    // earlier beam's)
    for (int i = threadIdx.x; i < n; i += NT) {
        const int w = i / a.kc, j = i - w * a.kc;
        if (j >= a.M)
            continue;
        const uint64_t key = score[i];
        int place = j;
        for (int o = 0; o < a.W && place < a.M; ++o) {
            if (o == w)
                continue;
            int lo = 0, hi = a.kc;  // first of o's list that does not go before
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                const uint64_t other = score[o * a.kc + mid];
                if (other > key || (other == key && o < w))
                    lo = mid + 1;
                else
                    hi = mid;
            }
            place += lo;
        }
        if (place < a.M) {
            const uint64_t u = (key >> 63) ? (key ^ (1ull << 63)) : ~key;
            s_score[place] = key == ~0ull ? __builtin_nan("") : __builtin_bit_cast(double, u);
            s_parent[place] = w;
            s_token[place] = token[i];
        }
    }
    __syncthreads();
    if (blockIdx.y == 0) {
        for (int j = threadIdx.x; j < a.M; j += NT) {
            const int64_t o = static_cast<int64_t>(b) * a.M + j;
            a.o_scores[o] = static_cast<float>(s_score[j]);
            a.o_parent[o] = s_parent[j];
            a.o_token[o] = s_token[j];
            if (a.o_finished)
                a.o_finished[o] = (a.finished && a.finished[b * a.W + s_parent[j]]) || s_token[j] == a.eos;
        }
        if (a.o_history)
            for (int i = threadIdx.x; i < a.M * a.T; i += NT) {
                const int j = i / a.T, t = i - j * a.T;
                a.o_history[static_cast<int64_t>(b) * a.M * a.T + i] =
                    t == a.step ? s_token[j]
                                : a.history[(static_cast<int64_t>(b) * a.W + s_parent[j]) * a.T + t];
            }
    }
    if (a.o_state) {
        const char *src = a.state + b * a.W * a.state_bytes;
        char *dst = a.o_state + b * a.M * a.state_bytes;
        if (a.state_bytes % 16 == 0)
            copy_rows<uint4>(src, dst, a.state_bytes, a.M, s_parent, blockIdx.y, gridDim.y);
        else
            copy_rows<uint32_t>(src, dst, a.state_bytes, a.M, s_parent, blockIdx.y, gridDim.y);
    }
}

}  // namespace DH_NS

namespace dhtop {

using namespace dht;

namespace {

constexpr int TARGET_BLOCKS = 1024;

int vec_len(int dtype) { return dtype == DOMINO_F32 ? 4 : 8; }

Split split_of(const domino_logits &lg, int k)
{
    const int64_t rows = static_cast<int64_t>(lg.B) * lg.R;
    const int nvec = (lg.V + vec_len(lg.dtype) - 1) / vec_len(lg.dtype);
    const int least = (nvec + NT * 16 - 1) / (NT * 16);
    int64_t n = rows ? (TARGET_BLOCKS + rows - 1) / rows : 1;
    n = n < nvec / NT ? n : nvec / NT;
    n = n < MERGE_LIST / k ? n : MERGE_LIST / k;
    n = n > least ? n : least;
    Split sp;
    sp.cvec = static_cast<int>((nvec + n - 1) / n);
    sp.nch = (nvec + sp.cvec - 1) / sp.cvec;
    sp.nv = 1;
    while (sp.nv * NT < sp.cvec)
        sp.nv *= 2;
    return sp;
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

template <typename T, int NV>
void launch_chunk(const Rows &rows, const Live &live, int k, const Split &sp, float tau, const TopOut &out,
                  unsigned grid, hipStream_t st)
{
    hipLaunchKernelGGL((k_top_chunk<T, NV>), dim3(grid), dim3(NT), 0, st, rows, live, k, sp.nch, sp.cvec,
                       scale_of(tau), 1.0 / static_cast<double>(tau), out);
}

template <typename T>
void pick_chunk(const Rows &rows, const Live &live, int k, const Split &sp, float tau, const TopOut &out,
                unsigned grid, hipStream_t st)
{
    if (sp.nv <= 2)
        launch_chunk<T, 2>(rows, live, k, sp, tau, out, grid, st);
    else if (sp.nv <= 4)
        launch_chunk<T, 4>(rows, live, k, sp, tau, out, grid, st);
    else if (sp.nv <= 8)
        launch_chunk<T, 8>(rows, live, k, sp, tau, out, grid, st);
    else
        launch_chunk<T, 16>(rows, live, k, sp, tau, out, grid, st);
}

struct Scratch {
    uint64_t *keys, *merged;
    Part *parts;
    size_t bytes;
};

Scratch scratch_of(const domino_logits &lg, int k, const Split &sp, void *ws)
{
    const size_t rows = static_cast<size_t>(lg.B) * lg.R, slots = rows * sp.nch;
    char *p = static_cast<char *>(ws);
    Scratch s;
    s.keys = reinterpret_cast<uint64_t *>(p);
    size_t at = round16(slots * k * sizeof(uint64_t));
    s.merged = reinterpret_cast<uint64_t *>(p + at);
    at += sp.nch > 1 ? round16(rows * k * sizeof(uint64_t)) : 0;
    s.parts = reinterpret_cast<Part *>(p + at);
    s.bytes = at + round16(slots * sizeof(Part));
    return s;
}

Rows rows_of(const domino_logits &lg, const int32_t *n_rows)
{
    Rows r;
    r.data = lg.data;
    r.bs = lg.batch_stride;
    r.rs = lg.row_stride;
    r.R = lg.R;
    r.V = lg.V;
    r.n_rows = n_rows;
    return r;
}

hipError_t select(const domino_logits &lg, const Rows &rows, const Live &live, int k, float tau, const Split &sp,
                  const TopOut &out, uint64_t *merged, hipStream_t st)
{
    const unsigned n = static_cast<unsigned>(lg.B) * static_cast<unsigned>(lg.R);
    if (lg.dtype == DOMINO_F32)
        pick_chunk<float>(rows, live, k, sp, tau, out, n * sp.nch, st);
    else
        pick_chunk<bf16s>(rows, live, k, sp, tau, out, n * sp.nch, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || sp.nch == 1)
        return e;
    hipLaunchKernelGGL(k_top_merge, dim3(n), dim3(NT), 0, st, rows, live, k, sp.nch, 1.0 / static_cast<double>(tau),
                       out, merged);
    return hipGetLastError();
}

}  // namespace

size_t workspace_bytes(const domino_logits &lg, int k)
{
    return scratch_of(lg, k, split_of(lg, k), nullptr).bytes;
}

hipError_t top(const domino_logits &lg, int k, float tau, const int32_t *n_rows, void *ws, int32_t *ids,
               float *values, float *lse, hipStream_t st)
{
    const Split sp = split_of(lg, k);
    const Scratch s = scratch_of(lg, k, sp, ws);
    const TopOut out = {s.keys, s.parts, ids, values, lse};
    return select(lg, rows_of(lg, n_rows), Live{nullptr, nullptr}, k, tau, sp, out, nullptr, st);
}

hipError_t beam(const domino_logits &lg, const domino_beam &bm, void *ws, hipStream_t st)
{
    const int kc = bm.n_out < lg.V ? bm.n_out : lg.V;
    const Split sp = split_of(lg, kc);
    const Scratch s = scratch_of(lg, kc, sp, ws);
    const TopOut out = {s.keys, s.parts, nullptr, nullptr, nullptr};
    const hipError_t e =
        select(lg, rows_of(lg, nullptr), Live{bm.scores, bm.finished}, kc, 1.f, sp, out, s.merged, st);
    if (e != hipSuccess)
        return e;
    BeamArgs a;
    a.W = lg.R, a.M = bm.n_out, a.V = lg.V, a.kc = kc, a.nch = sp.nch, a.eos = bm.eos, a.T = bm.T, a.step = bm.step;
    a.state_bytes = bm.state ? bm.state_bytes : 0;
    a.lists = sp.nch > 1 ? s.merged : s.keys;
    a.parts = s.parts;
    a.scores = bm.scores;
    a.finished = bm.finished;
    a.state = static_cast<const char *>(bm.state);
    a.history = bm.history;
    a.o_scores = bm.out_scores;
    a.o_parent = bm.out_parent;
    a.o_token = bm.out_token;
    a.o_finished = bm.out_finished;
    a.o_state = bm.state ? static_cast<char *>(bm.out_state) : nullptr;
    a.o_history = bm.history ? bm.out_history : nullptr;
    // a block of its own for every 16 KiB of state, at most 64 a batch entry
    int64_t parts = a.o_state ? (a.M * a.state_bytes + 16383) / 16384 : 1;
    parts = parts < 1 ? 1 : parts > 64 ? 64 : parts;
    const size_t lds = static_cast<size_t>(lg.R) * kc * (sizeof(uint64_t) + sizeof(int));
    hipLaunchKernelGGL(k_beam_merge, dim3(lg.B, static_cast<unsigned>(parts)), dim3(NT), lds, st, a);
    return hipGetLastError();
}

}  // namespace dhtop
