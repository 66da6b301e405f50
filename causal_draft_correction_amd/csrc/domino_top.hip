// The largest logits of vocabulary rows, and one step of beam search over them.
//
// top: for each row z of [B, R, V] logits the k largest (largest first; ties to the lowest id, NaN above every
// number, -0 == +0) and lse = log sum_v exp(z_v / tau).
//
// k_top_chunk reads a row once, one block per chunk (256 threads, at most 8 vectors each: 32 KiB), and leaves the
// chunk's k largest and its part of the sum.  The k-th largest of the threads' maxima bounds the k-th largest of the
// chunk from below; the waves' shares of it are found by ballots two bits at a time, 16 bits deep.  On rows in no
// particular order 1.5 k to 3 k elements reach the bound: their vectors go to LDS, from there they go to a list, and
// the place of each is the number of greater ones (of a list longer than 256, which is rare, by sorting it).
// k_top_merge joins the chunks' lists of a row in the same way; its bound is taken from the lists' heads.  A row that
// one block can hold (up to 1024 threads) is one chunk, and needs no join.
//
// What bounds it, on one MI355X: 512 bf16 rows of 151936, k = 20 (156 MB): 32.4 + 4.6 us, 4.8 TB/s in the chunks'
// launch, which issues 731 vector instructions a wave (59 of them exponentials, at 16 cycles, the others at 4): 30 us
// of issue at 2.4 GHz, so the vector units bound bfloat16, not the 24 us the bytes take.  float32 has half the elements
// a byte: 1024 rows of 50021, k = 16 (205 MB): 38 us in all, 5.4 TB/s.  Few rows are bound by latency: 17 f32 rows,
// k = 64: 8.8 + 5.6 us.
//
// Chunks of 8 vectors a thread against 16 (half the waves in flight): 34.3 against 35.8 us for the 512 rows.  More
// chunks a row give few rows more blocks, and the join more candidates: 17 rows, k = 64, 31 chunks 8.9 + 5.6 us,
// 61 chunks 10.4 + 5.4 us; so half as many blocks are aimed at for k > 32.
//
// beam: W beams' candidates score s_w + log softmax(z_w)_v.  Within a beam they are ordered by their logits, so the
// M best of all are among the M largest of each chunk, and k_top_chunk serves both.  k_beam_merge scores them in 64
// bits, ranks them as k_top_merge does, and writes state and history in the new order: 32 x 8 bf16 beams of 151936,
// 16 out of each, 4 KiB of state, one beam of each ended: 19.3 + 9.1 us (71 MB); its 2240 blocks with work are more than
// the 2048 that the device holds (8 a compute unit, by 61 registers and 20 KB of LDS), so the last 192 run almost alone.
// Four f32 beams of one request, 8 out: 5.2 + 8.2 us, latency.
//
// token log-probabilities with alternatives: the same launches (SCORE), which take the row's entropy with its sum and
// give the k largest as log-probabilities (dh_score.h).
#define DH_NT 256
#define DH_NS dht
#include "dh_rows.h"
#include "dh_score.h"
#include "dh_top.h"

#include <type_traits>

namespace DH_NS {

constexpr int VECS = 512;          // vectors of a chunk that LDS holds
constexpr int LIST = 1024;         // elements of a chunk that the LDS list holds
constexpr int MERGE_LIST = 4096;   // candidates of a row's chunks
constexpr int BEAM_LIST = 512;     // candidates of a beam step that are ranked by counting
constexpr int MAX_TIES = 128;      // places of the list kept for elements equal to the bound (at least MAX_K)
constexpr int COUNT_MAX = 256;     // up to here places are counted, above the list is sorted
constexpr int MAX_BEAMS = dhtop::MAX_W, MAX_OUT = dhtop::MAX_K;
static_assert(MAX_TIES >= dhtop::MAX_K, "the ties alone may be the result");
static_assert(LIST >= dhtop::MAX_K * 8, "a chunk of fewer vectors than k is taken whole");

// Rows that are not read: past n_rows; beams that are dead (score -inf), ended, or without a usable score.
struct Live {
    const float *scores;
    const uint8_t *finished;
};
__device__ inline bool row_live(const Rows &rows, const Live &lv, const Place &at)
{
    if (lv.scores) {
        const float s = lv.scores[at.row];
        return s > NEG_INF && s < -NEG_INF && !(lv.finished && lv.finished[at.row]);
    }
    return rows.counts(at.b, at.r);
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
constexpr uint32_t ORD_NEG_INF = 0x007FFFFFu;  // ord_f32(-inf)
__device__ inline uint32_t word(float f) { return __float_as_uint(f); }
__device__ inline uint32_t word(uint32_t u) { return u; }
__device__ inline float key_value(uint64_t key) { return unord_f32(static_cast<uint32_t>(key >> 32)); }

// The n-th largest of the wave's values with its bits below LAST cleared: at least n lanes reach it (0 if fewer
// than n hold more than 0).  Two bits a step, from bit FROM on where the n-th largest shares the bits above with the
// largest; all lanes get it.
template <int LAST, int FROM>
__device__ inline uint32_t wave_bound(uint32_t v, int n)
{
    static_assert(LAST % 2 == 0 && FROM % 2 == 0 && FROM <= 32, "two bits a step");
    uint32_t top = v;
    top = max(top, dpp_u32<DPP_QUAD_XOR1>(top));
    top = max(top, dpp_u32<DPP_QUAD_XOR2>(top));
    top = max(top, dpp_u32<DPP_HALF_MIRROR>(top));
    top = max(top, dpp_u32<DPP_ROW_MIRROR>(top));
    uint32_t a, b;
    row_pair_values(top, a, b);
    half_values(max(a, b), a, b);
    top = __builtin_amdgcn_readfirstlane(max(a, b));
    uint32_t t = 0;
    auto step = [&](int bit) {
        const uint32_t c1 = t | (1u << bit), c2 = t | (2u << bit), c3 = t | (3u << bit);
        const int n1 = __popcll(__ballot(v >= c1)), n2 = __popcll(__ballot(v >= c2)), n3 = __popcll(__ballot(v >= c3));
        t = n3 >= n ? c3 : n2 >= n ? c2 : n1 >= n ? c1 : t;
    };
    const uint32_t high = top >> FROM << FROM;
    if (__popcll(__ballot(v >= high)) >= n) {
        t = high;
    } else {
#pragma unroll
        for (int bit = 30; bit >= FROM; bit -= 2)
            step(bit);
    }
#pragma unroll
    for (int bit = FROM - 2; bit >= LAST; bit -= 2)
        step(bit);
    return t;
}

// A bound that at least n of the block's values reach: the lowest of the waves' bounds for their share of n.  `red`:
// one word a wave; one barrier.  All threads get the same.
template <int LAST, int FROM, int NTB>
__device__ inline uint32_t block_bound(uint32_t v, int n, uint32_t *red)
{
    constexpr int NW = NTB / 64;
    const uint32_t w = wave_bound<LAST, FROM>(v, (n + NW - 1) / NW);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = w;
    __syncthreads();
    uint32_t t = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i)
        t = t < red[i] ? t : red[i];
    return t;
}

// Places of the wave's hits in a list of the block, one atomic for all of them.
template <int N>
__device__ inline void wave_places(const bool (&hit)[N], int *count, int (&at)[N])
{
    int total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint64_t mask = __ballot(hit[i]);
        const uint32_t low = __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0);
        at[i] = total + static_cast<int>(__builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32), low));
        total += __popcll(mask);
    }
    if (total) {
        int base = 0;
        if ((threadIdx.x & 63) == 0)
            base = atomicAdd(count, total);
        base = __builtin_amdgcn_readfirstlane(base);
#pragma unroll
        for (int i = 0; i < N; ++i)
            at[i] += base;
    }
}

// Sorts list[0, n) in descending order; the list has room up to the next power of two.
template <int NTB>
__device__ inline void block_sort(uint64_t *list, int n)
{
    int len = 2;
    while (len < n)
        len <<= 1;
    for (int i = n + static_cast<int>(threadIdx.x); i < len; i += NTB)
        list[i] = 0;
    for (int size = 2; size <= len; size <<= 1)
        for (int step = size >> 1; step; step >>= 1) {
            __syncthreads();
            for (int i = threadIdx.x; i < len / 2; i += NTB) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const uint64_t x = list[a], y = list[b];
                if ((x < y) == ((a & size) == 0))
                    list[a] = y, list[b] = x;
            }
        }
    __syncthreads();
}

// Hands the k largest of list[0, n), n <= COUNT_MAX, to emit(place, key), largest first; places past n get key 0.
template <int NTB, typename F>
__device__ inline void emit_counted(uint64_t *list, int *place, int n, int k, F emit)
{
    // 2^shift threads take one key each, and NTB / 2^shift a slice of the others
    const int t = threadIdx.x, shift = n <= 64 ? 6 : n <= 128 ? 7 : 8;
    place[t] = 0;
    if (t == 0 && (n & 1))
        list[n] = 0;
    __syncthreads();
    const int i = t & ((1 << shift) - 1), slices = NTB >> shift, pairs = (n + 1) / 2;
    const int len = (pairs + slices - 1) / slices, j0 = (t >> shift) * len, j1 = j0 + len < pairs ? j0 + len : pairs;
    if (i < n) {
        const uint64_t key = list[i];
        const ulonglong2 *two = reinterpret_cast<const ulonglong2 *>(list);
        int above = 0;
#pragma unroll 4
        for (int j = j0; j < j1; ++j) {
            const ulonglong2 o = two[j];
            above += (o.x > key) + (o.y > key);
        }
        if (above)
            atomicAdd(&place[i], above);
    }
    __syncthreads();
    if (t < n && place[t] < k)
        emit(place[t], list[t]);
    for (int at = n + t; at < k; at += NTB)
        emit(at, 0ull);
}

// The same for longer lists (room up to the next power of two), which are sorted.
template <int NTB, typename F>
__device__ inline void emit_largest(uint64_t *list, int *place, int n, int k, F emit)
{
    if (n <= COUNT_MAX) {
        emit_counted<NTB>(list, place, n, k, emit);
    } else {
        block_sort<NTB>(list, n);
        for (int i = threadIdx.x; i < k; i += NTB)
            emit(i, list[i]);
    }
}

template <int NTB>
struct ChunkShared {
    alignas(16) uint64_t list[LIST];
    uint4 vec[VECS];
    int at[VECS];            // first element of each
    uint32_t bound[NTB / 64];
    int place[NTB];
    float m[NTB / 64];
    double s[NTB / 64], score[NTB / 64][2];
    uint32_t count[2 * (NTB / 64)];
    int nvec, n;
};

// The word by which argmax_key orders an element: NaN above +inf, -0 as +0.
__device__ inline uint32_t key_word(float f) { return static_cast<uint32_t>(argmax_key(f, 0) >> 32); }

// f(value, index, whether there is one) for the n elements at z, two vectors a thread at a time: more would halve the
// waves of the common path.
template <typename T, int NTB, typename F>
__device__ __forceinline__ void each(const T *z, int n, F f)
{
    typedef Vec<T> VT;
    constexpr int STEP = 2;
#pragma unroll 1
    for (int i = 0; i * STEP * NTB * VT::N < n; ++i) {
        typename VT::raw x[STEP];
        load_chunk<T, STEP, NTB, true>(x, z, n, i, STEP * NTB);
#pragma unroll
        for (int u = 0; u < STEP; ++u) {
            const int at = ((i * STEP + u) * NTB + static_cast<int>(threadIdx.x)) * VT::N;
#pragma unroll
            for (int e = 0; e < VT::N; ++e)
                f(VT::get(x[u], e), at + e, at + e < n);
        }
    }
}

// The sum of the threads' counts (at most 2^16 a wave, which float32 holds).  One barrier.  `count`: two rows of a word
// a wave, which calls take in turn, so that a row's words were read before the other one's barrier.
template <int NTB>
__device__ inline int block_count(int mine, int turn, uint32_t *count)
{
    const float all = wave_sum(static_cast<float>(mine));
    count += turn * (NTB / 64);
    if ((threadIdx.x & 63) == 0)
        count[threadIdx.x >> 6] = static_cast<uint32_t>(all);
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < NTB / 64; ++w)
        sum += static_cast<int>(count[w]);
    return sum;
}

// Narrows [lo, hi), of which at least k of a block's words reach lo and fewer than k reach hi, until at most `most`
// reach lo, or to one word.  reach(c): how many of the thread's words reach c.  Begins with row 0 of `count`.
template <int NTB, typename F>
__device__ __forceinline__ void bisect(uint64_t &lo, uint64_t &hi, int k, int most, uint32_t *count, F reach)
{
    for (int turn = 0; hi - lo > 1; turn ^= 1) {  // (at most 64 turns)
        const uint64_t c = lo + (hi - lo) / 2;
        const int n = block_count<NTB>(reach(c), turn, count);
        if (n < k)
            hi = c;
        else
            lo = c;
        if (n >= k && n <= most)
            break;
    }
}

// The next entries of the list, in the threads' order: those with `tie`, behind the greater ones and the `have` equal
// ones before them, up to place k.  Two barriers.
template <int NTB>
__device__ inline void list_ties(uint64_t *list, int greater, int &have, int k, bool tie, uint64_t key,
                                 uint32_t *count)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t mask = __ballot(tie);
    if (lane == 0)
        count[wave] = __popcll(mask);
    __syncthreads();
    int before = have, all = have;
#pragma unroll
    for (int w = 0; w < NTB / 64; ++w) {
        before += w < wave ? static_cast<int>(count[w]) : 0;
        all += static_cast<int>(count[w]);
    }
    const int at = greater + before + __popcll(mask & ((1ull << lane) - 1));
    if (tie && at < k)
        list[at] = key;
    have = all;
    __syncthreads();
}

// The elements whose words exceed t go to the list, as far as they have room; returns how many there are.
template <typename T, int NTB>
__device__ __forceinline__ int list_above(const T *z, int n, int v0, uint32_t t, ChunkShared<NTB> &sh)
{
    __syncthreads();
    if (threadIdx.x == 0)
        sh.n = 0;
    __syncthreads();
    each<T, NTB>(z, n, [&](float f, int i, bool in) {
        const bool one[1] = {in && key_word(f) > t};
        int to[1];
        wave_places(one, &sh.n, to);
        if (one[0] && to[0] < LIST - MAX_TIES)
            sh.list[to[0]] = argmax_key(f, static_cast<uint32_t>(v0 + i));
    });
    __syncthreads();
    return sh.n;
}

// The list of a chunk with any values: masked rows (most elements are -inf), sorted rows, few different values, NaN
// and infinities.  The elements above a bound go to the list, then those equal to it in the order of their ids until
// k are there.  `lo`: a bound that at least k elements reach (or all, where there are fewer); `hi`: one that none does.
// 16 f32 rows of 32000 with 2000 neighbours left by a mask, k = 64: 51 us a call, where 64 passes for a maximum each
// took 406; 512 rows of 151936 with a +inf each 64 us, instead of 425.
template <typename T, int NTB>
__device__ __forceinline__ void list_any(const T *row, int v0, int v1, int k, uint32_t lo, uint64_t hi,
                                         ChunkShared<NTB> &sh)
{
    uint32_t t = lo;
    int greater = 0;
#pragma unroll 1
    for (int attempt = 0; attempt < 2; ++attempt) {  // (the second has few enough)
        if (attempt) {
            uint64_t least = static_cast<uint64_t>(lo) + 1;
            bisect<NTB>(least, hi, k, LIST - MAX_TIES, sh.count, [&](uint64_t c) {
                int reach = 0;
                each<T, NTB>(row + v0, v1 - v0, [&](float f, int, bool in) { reach += in & (key_word(f) >= c); });
                return reach;
            });
            t = static_cast<uint32_t>(least);
        }
        greater = list_above(row + v0, v1 - v0, v0, t, sh);
        if (greater <= LIST - MAX_TIES)
            break;
        greater = LIST - MAX_TIES;  // (the list's length, whatever happens to the row meanwhile)
    }
    int have = 0;  // equal ones so far
    for (int base = v0; base < v1 && greater + have < k; base += NTB) {
        const int v = base + static_cast<int>(threadIdx.x);
        const float z = v < v1 ? Vec<T>::one(row + v) : 0.f;
        list_ties<NTB>(sh.list, greater, have, k, v < v1 && key_word(z) == t,
                       argmax_key(z, static_cast<uint32_t>(v)), sh.count);
    }
    if (threadIdx.x == 0)
        sh.n = greater + have < k ? greater + have : greater > k ? greater : k;
    __syncthreads();
}

// What one block leaves of its chunk: keys and part, or (a row of one chunk) the results.
struct TopOut {
    uint64_t *keys;    // [rows, nch, k]
    Part *parts;       // [rows, nch]
    int32_t *ids;      // [rows, k]; NULL where keys and parts are wanted
    float *values, *lse;
    ScorePart *score_parts;  // SCORE: in the place of parts; values are log-probabilities, lse is not there
    Score score;
};

template <bool SCORE>
__device__ inline bool row_wanted(const Rows &rows, const Live &live, const TopOut &o, const Place &at)
{
    if constexpr (SCORE)
        return score_counts(rows, o.score, at);
    return row_live(rows, live, at);
}

// The results of a row that is left out.
template <bool SCORE, int NTB>
__device__ inline void put_none(const TopOut &o, int row, int k)
{
    for (int i = threadIdx.x; i < k; i += NTB) {
        o.ids[static_cast<int64_t>(row) * k + i] = -1;
        o.values[static_cast<int64_t>(row) * k + i] = NEG_INF;
    }
    if (threadIdx.x == 0) {
        if constexpr (SCORE)
            no_score(o.score, row);
        else
            o.lse[row] = NEG_INF;
    }
}

__device__ inline void put_result(const TopOut &o, int row, int k, int place, uint64_t key)
{
    o.ids[static_cast<int64_t>(row) * k + place] = static_cast<int32_t>(key_index(key));
    o.values[static_cast<int64_t>(row) * k + place] = key_value(key);
}

__device__ inline void put_alternative(const TopOut &o, int row, int k, int place, uint64_t key, const ScorePart &all,
                                       double log_s, double inv_tau)
{
    o.ids[static_cast<int64_t>(row) * k + place] = static_cast<int32_t>(key_index(key));
    o.values[static_cast<int64_t>(row) * k + place] =
        static_cast<float>(log_prob(key_value(key), all, log_s, inv_tau));
}
__device__ inline float *stats_of(const Score &score, int row)
{
    return score.stats ? score.stats + static_cast<int64_t>(row) * SCORE_STATS : nullptr;
}

// One chunk of a row: its k largest and its part of the row's sum, or the row's results where it is one chunk.
template <typename T, int NTB, int NV, bool SCORE>
__global__ __launch_bounds__(NTB) void k_top_chunk(Rows rows, Live live, int k, Split sp, Scale sc,
                                                  double inv_tau, TopOut out)
{
    typedef Vec<T> VT;
    __shared__ ChunkShared<NTB> sh;
    const int nch = sp.nch, cvec = sp.cvec, i_row = static_cast<int>(sp.by.quotient(blockIdx.x));
    const int c = static_cast<int>(blockIdx.x) - i_row * nch;
    const Place place = rows.place(i_row);
    const int row = place.row;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const bool direct = nch == 1 && out.ids;
    if (!row_wanted<SCORE>(rows, live, out, place)) {
        if (direct)
            put_none<SCORE, NTB>(out, row, k);
        return;
    }
    const T *z = row_at<T>(rows, place);
    const int v0 = chunk_begin<T>(c, cvec, rows.V), v1 = chunk_begin<T>(c + 1, cvec, rows.V);
    typename VT::raw x[NV];
    load_chunk<T, NV, NTB>(x, z, rows.V, c, cvec);
    if (threadIdx.x == 0)
        sh.nvec = sh.n = 0;

    float vm[NV], tm = NEG_INF;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        vm[u] = VT::max_with(x[u], NEG_INF);
        tm = fmaxf(tm, vm[u]);
    }
    // the bound: a thread without an element counts as below everything
    const bool any = v0 + static_cast<int>(threadIdx.x) * VT::N < v1;
    const uint32_t top = any ? ord_f32(tm) : 0u;
    const float wm = wave_max(tm);
    if (lane == 0)
        sh.m[wave] = wm;
    const uint32_t t_ord = block_bound<16, 26, NTB>(top, k, sh.bound);
    float m = sh.m[0];
#pragma unroll
    for (int w = 1; w < NTB / 64; ++w)
        m = fmaxf(m, sh.m[w]);
    const float t = t_ord > ORD_NEG_INF ? unord_f32(t_ord) : NEG_INF;
    bool hit[NV];
    int at[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u)
        hit[u] = vm[u] >= t;  // (places past the chunk are told by their index)
    wave_places(hit, &sh.nvec, at);
#pragma unroll
    for (int u = 0; u < NV; ++u)
        if (hit[u] && at[u] < VECS) {
            sh.vec[at[u]] = make_uint4(word(x[u][0]), word(x[u][1]), word(x[u][2]), word(x[u][3]));
            sh.at[at[u]] = v0 + (u * NTB + static_cast<int>(threadIdx.x)) * VT::N;
        }
    const Expo ex(m > NEG_INF ? m : 0.f, sc);
    // (a thread's sum in float32, all others in 64 bits: continuations of different beams lie close to each other)
    ScorePart all = {};
    bool nan = false;
    if constexpr (SCORE) {
        all = block_score<T, NV, NTB>(x, z, rows.V, c, cvec, tm, m, sh.m, sh.score, ex, sc, nan);
    } else {
        const double s = wave_sum_f64(ex.small ? sum_exps<T, true>(x, ex, sc) : sum_exps<T, false>(x, ex, sc));
        if (lane == 0)
            sh.s[wave] = s;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NTB / 64; ++w)
            nan |= sh.s[w] != sh.s[w];
    }
    const int nvec = sh.nvec;
    // one element a thread
    if (nvec <= VECS)
        for (int i = threadIdx.x; i < (nvec * VT::N + 63) / 64 * 64; i += NTB) {
            const int j = i / VT::N, e = i % VT::N, v = j < nvec ? sh.at[j] + e : v1;
            const float f = VT::word_at(reinterpret_cast<const uint32_t *>(sh.vec), i);
            const bool one[1] = {v < v1 && f >= t};
            int to[1];
            wave_places(one, &sh.n, to);
            if (one[0] && to[0] < LIST)
                sh.list[to[0]] = argmax_key(f, static_cast<uint32_t>(v));
        }
    __syncthreads();
    const int64_t slot = static_cast<int64_t>(row) * nch + c;
    const double log_s = SCORE && direct ? log1p(all.s) : 0.0;
    auto emit = [&](int at, uint64_t key) {
        if (SCORE && direct)
            put_alternative(out, row, k, at, key, all, log_s, inv_tau);
        else if (direct)
            put_result(out, row, k, at, key);
        else
            out.keys[slot * k + at] = key;
    };
    const int n = sh.n;
    bool infinite = false;
    if (!nan && nvec <= VECS && n <= LIST) {
        emit_largest<NTB>(sh.list, sh.place, n, k, emit);
    } else {
        if (nan) {
            // NaN or +inf among the elements
            bool any_nan = false;
            for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += NTB) {
                const float f = VT::one(z + v);
                any_nan |= f != f;
            }
            nan = __syncthreads_or(any_nan);
            infinite = !nan;
        }
        const uint64_t hi = nan ? 1ull << 32 : static_cast<uint64_t>(key_word(m)) + 1;
        list_any(z, v0, v1, k, t_ord > ORD_NEG_INF ? t_ord : ORD_NEG_INF, hi, sh);
        emit_largest<NTB>(sh.list, sh.place, sh.n, k, emit);
    }
    if constexpr (SCORE) {
        if (threadIdx.x == NTB - 1) {
            if (direct)
                put_score(out.score, row, VT::one(z + out.score.tokens[row]), all, log_s, inv_tau,
                          stats_of(out.score, row));
            else
                out.score_parts[slot] = all;
        }
        return;
    }
    if (threadIdx.x == NTB - 1) {  // (of the wave with the least to rank)
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < NTB / 64; ++w)
            total += sh.s[w];
        total *= ex.fix(sc);
        const Part part = nan ? Part{__builtin_nanf(""), 1.0} : infinite ? Part{-NEG_INF, 1.0} : Part{m, total};
        if (direct)
            out.lse[row] = part.m == NEG_INF ? NEG_INF
                           : nan || infinite ? part.m
                                             : static_cast<float>(part.m * inv_tau + log(total));
        else
            out.parts[slot] = part;
    }
}

struct MergeShared {
    alignas(16) uint64_t list[MERGE_LIST];
    uint32_t bound[NWAVE];
    int place[NT];
    uint32_t count[2 * NWAVE];
    int n;
};

// How many of the thread's keys have a word above t.
template <int PER>
__device__ inline int above(const uint64_t (&keys)[PER], uint32_t t)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        n += static_cast<uint32_t>(keys[i] >> 32) > t;
    return n;
}

// The candidates of nch sorted lists of k keys that reach the k-th largest of the lists' heads go to sh.list;
// returns how many.  A thread takes PER keys; q heads of each list, one a thread (of more than NT lists, the first
// NT heads).
template <int PER>
__device__ inline int merge_list(const uint64_t *keys, int nch, int k, MergeShared &sh)
{
    const int lane = threadIdx.x & 63, n = nch * k;
    uint64_t mine[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = i * NT + static_cast<int>(threadIdx.x);
        mine[i] = at < n ? keys[at] : 0;
    }
    int q = NT / nch;
    q = q < 1 ? 1 : q < k ? q : k;
    // head h: place h / nch of list h % nch, dealt out over the waves
    const int h = lane * NWAVE + (static_cast<int>(threadIdx.x) >> 6), r = h / nch;
    const uint32_t head = r < q ? static_cast<uint32_t>(keys[static_cast<int64_t>(h - r * nch) * k + r] >> 32) : 0;
    if (threadIdx.x == 0)
        sh.n = 0;
    const uint32_t t = block_bound<12, 26, NT>(head, k, sh.bound);
    bool hit[PER];
    int at[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        hit[i] = static_cast<uint32_t>(mine[i] >> 32) >= t && mine[i];
    wave_places(hit, &sh.n, at);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (hit[i])
            sh.list[at[i]] = mine[i];
    __syncthreads();
    const int all = sh.n;
    if (all <= COUNT_MAX)
        return all;
    // Too many to count places: mostly equal ones (what a mask left out).  A bound that fewer exceed, then those equal
    // to it in the order of the lists, which is that of their ids.  16 f32 rows of 151936 with 6000 neighbours left by
    // a mask, k = 128: 24 us a call, where a sorted list took 91.
    uint64_t lo = t > ORD_NEG_INF ? t : ORD_NEG_INF, hi = 1ull << 32;
    int greater = block_count<NT>(above<PER>(mine, static_cast<uint32_t>(lo)), 1, sh.count);
    if (greater > COUNT_MAX)
        bisect<NT>(++lo, hi, k, COUNT_MAX, sh.count,
                   [&](uint64_t c) { return above<PER>(mine, static_cast<uint32_t>(c - 1)); });
    const uint32_t u = static_cast<uint32_t>(lo);
    __syncthreads();
    if (threadIdx.x == 0)
        sh.n = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        hit[i] = static_cast<uint32_t>(mine[i] >> 32) > u;
    wave_places(hit, &sh.n, at);
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (hit[i])
            sh.list[at[i]] = mine[i];
    __syncthreads();
    greater = sh.n;
    int have = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (greater + have < k)
            list_ties<NT>(sh.list, greater, have, k, static_cast<uint32_t>(mine[i] >> 32) == u, mine[i], sh.count);
    return greater + have < k ? greater + have : greater > k ? greater : k;
}

// The k largest of a row from its chunks' lists, and its log-sum-exp (TS: with the token's log-probability and the
// entropy, of logits of this type).
template <int PER, typename TS = void>
__global__ __launch_bounds__(NT) void k_top_merge(Rows rows, Live live, int k, int nch, double inv_tau, TopOut out)
{
    constexpr bool SCORE = !std::is_void<TS>::value;
    __shared__ MergeShared sh;
    const Place place = rows.place(blockIdx.x);
    const int row = place.row;
    if (!row_wanted<SCORE>(rows, live, out, place)) {
        put_none<SCORE, NT>(out, row, k);
        return;
    }
    const int64_t slot = static_cast<int64_t>(row) * nch;
    if constexpr (SCORE) {
        const ScorePart *parts = out.score_parts + slot, first = first_part(parts, nch);
        const float z = Vec<TS>::one(row_at<TS>(rows, place) + out.score.tokens[row]);
        const int n = merge_list<PER>(out.keys + slot * k, nch, k, sh);
        const ScorePart all = join_parts(first, parts, nch, inv_tau);
        const double log_s = log1p(all.s);
        emit_counted<NT>(sh.list, sh.place, n, k, [&](int at, uint64_t key) {
            put_alternative(out, row, k, at, key, all, log_s, inv_tau);
        });
        if (threadIdx.x == NT - 1)
            put_score(out.score, row, z, all, log_s, inv_tau, stats_of(out.score, row));
        return;
    }
    const Part part = first_part(out.parts + slot, nch);
    const int n = merge_list<PER>(out.keys + slot * k, nch, k, sh);
    emit_counted<NT>(sh.list, sh.place, n, k, [&](int at, uint64_t key) { put_result(out, row, k, at, key); });
    if (threadIdx.x >= NT - 64) {  // the wave with the least to rank
        float m;
        double s;
        join_parts(part, out.parts + slot, nch, inv_tau, m, s);
        if (threadIdx.x == NT - 1)
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
    const uint64_t *keys;    // [B * W, nch, kc]: the largest logits of each chunk, largest first
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

// Part `part` of nparts of the M rows of `bytes` bytes each, row j from src's row parent[j]; four loads in flight.
template <typename V>
__device__ inline void copy_rows(const char *src, char *dst, int64_t bytes, int M, const int *parent, int part,
                                 int nparts)
{
    const int64_t per = bytes / static_cast<int64_t>(sizeof(V)), all = per * M;
    const int64_t stride = static_cast<int64_t>(nparts) * blockDim.x;
    const bool narrow = all + 4 * stride <= 0x7FFFFFFF;
    for (int64_t i0 = static_cast<int64_t>(part) * blockDim.x + threadIdx.x; i0 < all; i0 += 4 * stride) {
        V v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + u * stride < all ? i0 + u * stride : all - 1;
            const int64_t j = narrow ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per) : i / per;
            v[u] = reinterpret_cast<const V *>(src)[parent[j] * per + (i - j * per)];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + u * stride < all)
                reinterpret_cast<V *>(dst)[i0 + u * stride] = v[u];
    }
}

// A candidate: its score's word, its beam, and its place among that beam's candidates (larger: earlier; a live
// beam's key, or the complement of the place).
struct Cand {
    uint64_t score, place;
    int w;
};
__device__ inline bool before(const Cand &a, const Cand &b)
{
    // (no branches)
    return (a.score > b.score) | ((a.score == b.score) & ((a.w < b.w) | ((a.w == b.w) & (a.place > b.place))));
}
enum { LIVE, DEAD, ENDED, BAD };
constexpr uint64_t ORD64_NEG_INF = 0x000FFFFFFFFFFFFFull;  // ord_f64(-inf)

struct BeamShared {
    Cand list[BEAM_LIST];
    int place[BEAM_LIST];
    uint32_t bound[16], count[2 * 16];
    uint64_t top[16];
    int tie[MAX_BEAMS];
    double score[MAX_BEAMS], log_s[MAX_BEAMS];
    float max[MAX_BEAMS];
    int kind[MAX_BEAMS];
    double o_score[MAX_OUT];
    int o_parent[MAX_OUT], o_token[MAX_OUT];
    int n;
};

__device__ inline double cand_score(const BeamShared &sh, int w, uint64_t key)
{
    const double z = key_value(key);
    // (z - max first: a row at the type's lowest value keeps its differences)
    return z == static_cast<double>(NEG_INF) ? z
                                             : sh.score[w] + ((z - static_cast<double>(sh.max[w])) - sh.log_s[w]);
}

__device__ inline void put_beam(BeamShared &sh, const BeamArgs &a, int i, const Cand &c)
{
    const uint64_t u = (c.score >> 63) ? (c.score ^ (1ull << 63)) : ~c.score;
    sh.o_score[i] = c.score == ~0ull ? __builtin_nan("") : __builtin_bit_cast(double, u);
    sh.o_parent[i] = c.w;
    int tok = static_cast<int>(key_index(c.place));
    if (sh.kind[c.w] == ENDED)  // the end token, then the others
        tok = tok == 0 ? a.eos : (tok - 1 < a.eos ? tok - 1 : tok);
    sh.o_token[i] = tok;
}

// The list for any mixture of dead, ended and live beams, NaN, equal scores and -inf, where the bound leaves fewer than
// M or too many: the candidates up to a score that at least M reach and at most BEAM_LIST, or up to the M-th of all, by
// bisection of the scores, then of the places within the beam that the M-th belongs to.  Returns how many.
// live(f): f(score, place, w) for the thread's candidates of live beams; beam(w, f): for those of beam w.  `kind`,
// `first`: of beam threadIdx.x, and its only candidate's score where it has ended; n candidates reach `bound`; `top`:
// the thread's best.  32 x 8 beams of 32000 f32, all of them ended, 16 out: 22 us a call, where 16 passes for the best
// one each took 85; 4 x 32 of 151936 with 3 tokens left by a mask, 128 out: 331 us instead of 5264.  Slow where wide beams
// hold many equal candidates: with PER = 0 every turn reads and scores all of them again (up to 64 turns for the score,
// up to 64 more for the place): 32 f32 beams of 151936 equal logits, 128 out, 2.2 ms; 16 beams, 64 out, 0.97 ms; 8 beams,
// 16 out, 0.3 ms; without equal ones 134, 58 and 24 us.
template <int NTB, typename L, typename O>
__device__ __forceinline__ int list_any_beams(const BeamArgs &a, int kind, uint64_t first, bool odd, int n,
                                              uint64_t bound, uint64_t top, BeamShared &sh, L live, O beam)
{
    const bool own = threadIdx.x < a.W;
    const int kc = a.kc;  // candidates of a beam that is not live, the same score for all (but the ended one's first)
    auto reach = [&](uint64_t c) {
        int r = 0;
        live([&](uint64_t score, uint64_t, int) { r += score >= c; });
        if (own && kind != LIVE)
            r += kind == BAD || ORD64_NEG_INF >= c ? kc : kind == ENDED && first >= c;
        return r;
    };
    uint64_t lo = ORD64_NEG_INF, hi = ~0ull;  // (NaN is ~0)
    if (odd) {
        if (block_count<NTB>(reach(hi), 1, sh.count) >= a.M)
            lo = hi;
    } else if (n < a.M) {
        hi = lo + 1;
    } else {  // from the bound that too many reach to the best
        lo = bound > lo ? bound : lo;
        top = wave_max_u64(top);
        if ((threadIdx.x & 63) == 0)
            sh.top[threadIdx.x >> 6] = top;
        __syncthreads();
        for (int w = 0; w < NTB / 64; ++w)
            top = max_u64(top, sh.top[w]);
        hi = top + 1;
    }
    bisect<NTB>(lo, hi, a.M, BEAM_LIST, sh.count, reach);
    const uint64_t t = lo;
    // of the candidates that score t, those of beams before `last` are in, and its own from place p on
    uint64_t p = 0;
    int last = a.W;
    if (hi - lo <= 1) {
        __syncthreads();
        if (own)
            sh.tie[threadIdx.x] = 0;
        __syncthreads();
        live([&](uint64_t score, uint64_t, int w) {
            if (score == t)
                atomicAdd(&sh.tie[w], 1);
        });
        if (own && kind != LIVE)
            sh.tie[threadIdx.x] = kind == BAD            ? kc * (t == ~0ull)
                                  : t == ORD64_NEG_INF ? kc - (kind == ENDED)
                                                       : kind == ENDED && first == t;
        int need = a.M - block_count<NTB>(t == ~0ull ? 0 : reach(t + 1), 1, sh.count);
        for (last = 0; last < a.W - 1 && sh.tie[last] < need; ++last)
            need -= sh.tie[last];
        if (sh.kind[last] == LIVE) {
            uint64_t end = ~0ull;
            if (sh.tie[last] > need)
                bisect<NTB>(p, end, need, need, sh.count, [&](uint64_t c) {
                    int r = 0;
                    beam(last, [&](uint64_t score, uint64_t place, int) { r += score == t && place >= c; });
                    return r;
                });
        } else {
            const int j0 = sh.kind[last] == ENDED && t == ORD64_NEG_INF;
            p = 0xFFFFFFFFu - static_cast<uint32_t>(j0 + need - 1);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0)
        sh.n = 0;
    __syncthreads();
    auto take = [&](uint64_t score, uint64_t place, int w) {
        if (score > t || (score == t && (w < last || (w == last && place >= p)))) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < BEAM_LIST)
                sh.list[at] = Cand{score, place, w};
        }
    };
    live(take);
    for (int w = 0; w < a.W; ++w)
        if (sh.kind[w] != LIVE)
            for (int j = threadIdx.x; j < kc; j += NTB)
                take(sh.kind[w] == BAD ? ~0ull
                                       : sh.kind[w] == ENDED && j == 0 ? ord_f64(sh.score[w]) : ORD64_NEG_INF,
                     0xFFFFFFFFu - static_cast<uint32_t>(j), w);
    __syncthreads();
    return sh.n < BEAM_LIST ? sh.n : BEAM_LIST;
}

// One batch entry.  Its blocks (blockIdx.y) all rank the candidates and share the copying of the state; block 0
// writes the rest.  The bound is the M-th largest of the threads' maxima, the candidates given out by their place
// in the chunks' lists: the threads hold the heads of the lists.  PER > 0: a thread holds its (at most PER) keys in
// registers, loaded before anything else is known; 0: any number, read twice.
template <int NTB, int PER>
__global__ __launch_bounds__(NTB) void k_beam_merge(BeamArgs a)
{
    __shared__ BeamShared sh;
    const int b = blockIdx.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int lists = a.W * a.nch, n_cand = lists * a.kc;
    const uint64_t *keys = a.keys + static_cast<int64_t>(b) * n_cand;
    // threads are dealt out over the waves.  PER > 0: thread i takes places i / lists + j * deep, j < PER, of list
    // i % lists.  PER = 0: candidate i is place i / lists of list i % lists.
    const int at0 = lane * (NTB / 64) + wave;
    const int deep = NTB / lists, r0 = at0 / lists, l0 = at0 - r0 * lists, w0 = l0 / a.nch;
    auto key_at = [&](int i, int &w) {
        const int r = i / lists, l = i - r * lists;
        w = l / a.nch;
        return keys[static_cast<int64_t>(l) * a.kc + r];
    };
    uint64_t mine[PER ? PER : 1], score[PER ? PER : 1];
    if constexpr (PER > 0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int r = r0 + j * deep;
            mine[j] = r0 < deep && r < a.kc ? keys[static_cast<int64_t>(l0) * a.kc + r] : 0;
        }
    }
    for (int w = wave; w < a.W; w += NTB / 64) {
        const int row = b * a.W + w;
        const Part *parts = a.parts + static_cast<int64_t>(row) * a.nch;
        const Part part = first_part(parts, a.nch);
        const float s = a.scores[row];
        const bool ended = a.finished && a.finished[row];
        int kind = s == NEG_INF ? DEAD : ended ? ENDED : s < -NEG_INF ? LIVE : BAD;
        if (kind == LIVE) {
            float m;
            double t;
            join_parts(part, parts, a.nch, 1.0, m, t);
            if (!(m < -NEG_INF))
                kind = BAD;
            if (lane == 0)
                sh.max[w] = m, sh.log_s[w] = log(t);
        }
        if (lane == 0)
            sh.kind[w] = kind, sh.score[w] = s;
    }
    if (threadIdx.x == 0)
        sh.n = 0;
    __syncthreads();
    const bool own = threadIdx.x < a.W;
    const int kind = own ? sh.kind[threadIdx.x] : DEAD;
    const double own_score = own ? sh.score[threadIdx.x] : 0.0;
    const uint64_t ended = kind == ENDED ? ord_f64(own_score) : 0;
    auto word_of = [&](uint64_t key, int w) {
        return key && sh.kind[w] == LIVE ? ord_f64(cand_score(sh, w, key)) : 0;
    };
    uint64_t top = ended;
    if constexpr (PER > 0) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            score[j] = word_of(mine[j], w0);
            top = max_u64(top, score[j]);
        }
    } else {
        for (int i = at0; i < n_cand; i += NTB) {
            int w;
            const uint64_t key = key_at(i, w);
            top = max_u64(top, word_of(key, w));
        }
    }
    const bool odd = __syncthreads_or(kind == BAD || (kind == ENDED && own_score != own_score));
    const uint32_t t = block_bound<8, 22, NTB>(static_cast<uint32_t>(top >> 32), a.M, sh.bound);
    auto take = [&](uint64_t score, uint64_t place, int w) {
        if (static_cast<uint32_t>(score >> 32) >= t && score > ORD64_NEG_INF) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < BEAM_LIST)
                sh.list[at] = Cand{score, place, w};
        }
    };
    if constexpr (PER > 0) {
        bool hit[PER];
        int at[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j)
            hit[j] = static_cast<uint32_t>(score[j] >> 32) >= t && score[j] > ORD64_NEG_INF;
        wave_places(hit, &sh.n, at);
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (hit[j] && at[j] < BEAM_LIST)
                sh.list[at[j]] = Cand{score[j], mine[j], w0};
    } else {
        for (int i = at0; i < n_cand; i += NTB) {
            int w;
            const uint64_t key = key_at(i, w);
            take(word_of(key, w), key, w);
        }
    }
    take(ended, 0xFFFFFFFFull, static_cast<int>(threadIdx.x));
    __syncthreads();
    int n = sh.n;
    if (odd || n < a.M || n > BEAM_LIST) {
        auto live = [&](auto f) {
            if constexpr (PER > 0) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (score[j])
                        f(score[j], mine[j], w0);
            } else {
                for (int i = at0; i < n_cand; i += NTB) {
                    int w;
                    const uint64_t key = key_at(i, w), word = word_of(key, w);
                    if (word)
                        f(word, key, w);
                }
            }
        };
        auto beam = [&](int w, auto f) {
            if constexpr (PER > 0) {
                if (w == w0)
                    live(f);
            } else {
                for (int i = threadIdx.x; i < a.nch * a.kc; i += NTB) {
                    const uint64_t key = keys[static_cast<int64_t>(w) * a.nch * a.kc + i], word = word_of(key, w);
                    if (word)
                        f(word, key, w);
                }
            }
        };
        n = list_any_beams<NTB>(a, kind, ended, odd, n, static_cast<uint64_t>(t) << 32, top, sh, live, beam);
    }
    // 2^shift threads take one candidate each, and NTB / 2^shift a slice of the others
    const int shift = n <= 32 ? 5 : n <= 64 ? 6 : n <= 128 ? 7 : n <= 256 ? 8 : 9;
    const int i = threadIdx.x & ((1 << shift) - 1), slices = NTB >> shift, len = (n + slices - 1) / slices;
    const int j0 = (threadIdx.x >> shift) * len, j1 = j0 + len < n ? j0 + len : n;
    if (threadIdx.x < BEAM_LIST)
        sh.place[threadIdx.x] = 0;
    __syncthreads();
    if (i < n) {
        const Cand c = sh.list[i];
        int place = 0;
#pragma unroll 2
        for (int j = j0; j < j1; ++j)
            place += before(sh.list[j], c);
        if (place)
            atomicAdd(&sh.place[i], place);
    }
    __syncthreads();
    if (threadIdx.x < n && sh.place[threadIdx.x] < a.M)
        put_beam(sh, a, sh.place[threadIdx.x], sh.list[threadIdx.x]);
    __syncthreads();
    if (blockIdx.y == 0) {
        for (int j = threadIdx.x; j < a.M; j += NTB) {
            const int64_t o = static_cast<int64_t>(b) * a.M + j;
            a.o_scores[o] = static_cast<float>(sh.o_score[j]);
            a.o_parent[o] = sh.o_parent[j];
            a.o_token[o] = sh.o_token[j];
            if (a.o_finished)
                a.o_finished[o] = (a.finished && a.finished[b * a.W + sh.o_parent[j]]) || sh.o_token[j] == a.eos;
        }
        if (a.o_history)
            for (int64_t i = threadIdx.x; i < static_cast<int64_t>(a.M) * a.T; i += NTB) {
                const int j = static_cast<int>(i / a.T), at = static_cast<int>(i - static_cast<int64_t>(j) * a.T);
                a.o_history[static_cast<int64_t>(b) * a.M * a.T + i] =
                    at == a.step ? sh.o_token[j]
                                 : a.history[(static_cast<int64_t>(b) * a.W + sh.o_parent[j]) * a.T + at];
            }
    }
    if (a.o_state) {
        const char *src = a.state + static_cast<int64_t>(b) * a.W * a.state_bytes;
        char *dst = a.o_state + static_cast<int64_t>(b) * a.M * a.state_bytes;
        if (a.state_bytes % 16 == 0)
            copy_rows<Vec<bf16s>::raw>(src, dst, a.state_bytes, a.M, sh.o_parent, blockIdx.y, gridDim.y);
        else
            copy_rows<uint32_t>(src, dst, a.state_bytes, a.M, sh.o_parent, blockIdx.y, gridDim.y);
    }
}

}  // namespace DH_NS

namespace dhtop {

using namespace dht;

namespace {

constexpr int TARGET_BLOCKS = 1024;           // aimed at where there are few rows
constexpr int MAX_NV = 8, LAST_NV = 16;       // vectors a thread takes at most; where the join would overflow

int vec_len(int dtype) { return dtype == DOMINO_F32 ? 4 : 8; }

// Rows that need no join: of up to 8 vectors for each of 256 threads, or of 1024 where every row has a compute unit for
// itself.  64 f32 rows of 32000, k = 8: 12.5 us a call and 9.0 us of kernel, split and joined 16.2 us and two kernels
// of 17 us from the first one's start to the second one's end; 1024 rows 27.3 us either way.  Beams are joined with
// each other in any case, and split rows reach that sooner.
bool whole_rows(int64_t rows, int nvec, bool for_beams)
{
    return !for_beams && (nvec <= NT * MAX_NV || (nvec <= 1024 * MAX_NV && rows <= 256));
}

Split split_of(const domino_logits &lg, int k, bool for_beams)
{
    const int64_t rows = static_cast<int64_t>(lg.B) * lg.R;
    const int nvec = (lg.V + vec_len(lg.dtype) - 1) / vec_len(lg.dtype);
    if (whole_rows(rows, nvec, for_beams))
        return split(nvec, 1);
    int least = (nvec + NT * MAX_NV - 1) / (NT * MAX_NV);
    if (least * k > MERGE_LIST)  // long rows and many logits of each: larger chunks
        least = (nvec + NT * LAST_NV - 1) / (NT * LAST_NV);
    // few rows are split over more blocks; each block costs the join its k candidates
    const int blocks = k > 32 ? TARGET_BLOCKS / 2 : TARGET_BLOCKS;
    int64_t n = rows ? (blocks + rows - 1) / rows : 1;
    n = n < nvec / (2 * NT) ? n : nvec / (2 * NT);
    n = n < MERGE_LIST / k ? n : MERGE_LIST / k;
    n = n < 64 ? n : 64;  // (a wave joins the parts of 64 at once)
    n = n > least ? n : least;
    return split(nvec, n);
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

template <typename T, int NTB, int NV>
void launch_chunk(const Rows &rows, const Live &live, int k, const Split &sp, double tau, const TopOut &out,
                  unsigned grid, hipStream_t st)
{
    if (out.score.tokens)
        hipLaunchKernelGGL((k_top_chunk<T, NTB, NV, true>), dim3(grid), dim3(NTB), 0, st, rows, live, k, sp,
                           scale_of(tau), 1.0 / tau, out);
    else
        hipLaunchKernelGGL((k_top_chunk<T, NTB, NV, false>), dim3(grid), dim3(NTB), 0, st, rows, live, k, sp,
                           scale_of(tau), 1.0 / tau, out);
}

template <typename T>
void pick_chunk(const Rows &rows, const Live &live, int k, const Split &sp, double tau, const TopOut &out,
                unsigned grid, hipStream_t st)
{
    // (one chunk a row: up to 1024 threads; else blocks of 256, which wait less for their own phases)
    if (sp.nv <= 2)
        launch_chunk<T, 256, 2>(rows, live, k, sp, tau, out, grid, st);
    else if (sp.nv <= 4)
        launch_chunk<T, 256, 4>(rows, live, k, sp, tau, out, grid, st);
    else if (sp.nv <= 8)
        launch_chunk<T, 256, 8>(rows, live, k, sp, tau, out, grid, st);
    else if (sp.nch > 1) {
        if constexpr (Vec<T>::N == 4)  // (split_of gives bfloat16 rows no such chunks)
            launch_chunk<T, 256, 16>(rows, live, k, sp, tau, out, grid, st);
    } else if (sp.nv <= 16)
        launch_chunk<T, 512, 8>(rows, live, k, sp, tau, out, grid, st);
    else
        launch_chunk<T, 1024, 8>(rows, live, k, sp, tau, out, grid, st);
}

struct Scratch {
    uint64_t *keys;
    void *parts;
    size_t bytes;
};

Scratch scratch_of(const domino_logits &lg, int k, const Split &sp, void *ws, size_t part = sizeof(Part))
{
    const size_t rows = static_cast<size_t>(lg.B) * lg.R, slots = rows * sp.nch;
    char *p = static_cast<char *>(ws);
    Scratch s;
    s.keys = reinterpret_cast<uint64_t *>(p);
    const size_t at = round16(slots * k * sizeof(uint64_t));
    s.parts = p + at;
    s.bytes = at + round16(slots * part);
    return s;
}

void chunks(const domino_logits &lg, const Rows &rows, const Live &live, int k, double tau, const Split &sp,
            const TopOut &out, hipStream_t st)
{
    const unsigned n = static_cast<unsigned>(lg.B) * static_cast<unsigned>(lg.R);
    if (lg.dtype == DOMINO_F32)
        pick_chunk<float>(rows, live, k, sp, tau, out, n * sp.nch, st);
    else
        pick_chunk<bf16s>(rows, live, k, sp, tau, out, n * sp.nch, st);
}

static_assert((dhtop::MAX_V / 4 + NT * LAST_NV - 1) / (NT * LAST_NV) * dhtop::MAX_K <= MERGE_LIST,
              "the candidates of the longest row fit one block's list");
static_assert((dhtop::MAX_V / 8 + NT * MAX_NV - 1) / (NT * MAX_NV) * dhtop::MAX_K <= MERGE_LIST,
              "bfloat16 rows are never cut into chunks of more than MAX_NV vectors a thread");

}  // namespace

size_t workspace_bytes(const domino_logits &lg, int k, bool for_beams)
{
    const Split sp = split_of(lg, k, for_beams);
    return sp.nch == 1 && !for_beams ? 0 : scratch_of(lg, k, sp, nullptr).bytes;
}

size_t score_workspace_bytes(const domino_logits &lg, int k)
{
    const Split sp = split_of(lg, k, false);
    return sp.nch == 1 ? 0 : scratch_of(lg, k, sp, nullptr, sizeof(ScorePart)).bytes;
}

namespace {

// The launches of top() and scores().
hipError_t largest(const domino_logits &lg, int k, double tau, const int32_t *n_rows, const TopOut &out, const Split &sp,
                   hipStream_t st)
{
    if (sp.nch > 1 && sp.nch > MERGE_LIST / k)  // (split_of makes no such split; the join would drop candidates)
        return hipErrorInvalidValue;
    const Rows rows = rows_of(lg, n_rows, n_rows != nullptr);
    const Live live = {nullptr, nullptr};
    chunks(lg, rows, live, k, tau, sp, out, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || sp.nch == 1)
        return e;
    const dim3 grid(static_cast<unsigned>(lg.B) * static_cast<unsigned>(lg.R));
    const double inv_tau = 1.0 / tau;
    const auto merge = [&](auto few, auto many) {
        if (sp.nch * k <= NT * 4)
            hipLaunchKernelGGL(few, grid, dim3(NT), 0, st, rows, live, k, sp.nch, inv_tau, out);
        else
            hipLaunchKernelGGL(many, grid, dim3(NT), 0, st, rows, live, k, sp.nch, inv_tau, out);
    };
    if (!out.score.tokens)
        merge(k_top_merge<4>, k_top_merge<MERGE_LIST / NT>);
    else if (lg.dtype == DOMINO_F32)
        merge(k_top_merge<4, float>, k_top_merge<MERGE_LIST / NT, float>);
    else
        merge(k_top_merge<4, bf16s>, k_top_merge<MERGE_LIST / NT, bf16s>);
    return hipGetLastError();
}

}  // namespace

hipError_t top(const domino_logits &lg, int k, double tau, const int32_t *n_rows, void *ws, int32_t *ids,
               float *values, float *lse, hipStream_t st)
{
    const Split sp = split_of(lg, k, false);
    const Scratch s = scratch_of(lg, k, sp, ws);
    const TopOut out = {s.keys, static_cast<Part *>(s.parts), ids, values, lse, nullptr, Score{}};
    return largest(lg, k, tau, n_rows, out, sp, st);
}

hipError_t scores(const domino_logits &lg, const dhtoken::Scores &want, int k, double tau, const int32_t *n_rows,
                  void *ws, int32_t *ids, float *logprobs, hipStream_t st)
{
    const Split sp = split_of(lg, k, false);
    const Scratch s = scratch_of(lg, k, sp, ws, sizeof(ScorePart));
    const TopOut out = {s.keys, nullptr, ids, logprobs, nullptr, static_cast<ScorePart *>(s.parts),
                        Score{want.tokens, want.logprob, want.entropy, want.stats}};
    return largest(lg, k, tau, n_rows, out, sp, st);
}

hipError_t beam(const domino_logits &lg, const domino_beam &bm, void *ws, hipStream_t st)
{
    const int kc = bm.n_out < lg.V ? bm.n_out : lg.V;
    const Split sp = split_of(lg, kc, true);
    const Scratch s = scratch_of(lg, kc, sp, ws);
    const TopOut out = {s.keys, static_cast<Part *>(s.parts), nullptr, nullptr, nullptr, nullptr, Score{}};
    chunks(lg, rows_of(lg, nullptr, true), Live{bm.scores, bm.finished}, kc, 1.f, sp, out, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    BeamArgs a;
    a.W = lg.R, a.M = bm.n_out, a.V = lg.V, a.kc = kc, a.nch = sp.nch, a.eos = bm.eos, a.T = bm.T, a.step = bm.step;
    a.state_bytes = bm.state ? bm.state_bytes : 0;
    a.keys = s.keys;
    a.parts = static_cast<const Part *>(s.parts);
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
    // a block of its own for every 16 KiB of state, at most 64 a batch entry: each ranks the candidates itself, which
    // takes less time than a launch of its own for the copies (4 us)
    int64_t parts = a.o_state ? (a.M * a.state_bytes + 16383) / 16384 : 1;
    parts = parts < 1 ? 1 : parts > 64 ? 64 : parts;
    const dim3 grid(lg.B, static_cast<unsigned>(parts));
    // places a thread of a block of 512 takes of its list
    const int lists = a.W * sp.nch, deep = lists <= 512 ? 512 / lists : 0;
    const int per = deep ? (kc + deep - 1) / deep : 1 << 30;
    if (per <= 2)
        hipLaunchKernelGGL((k_beam_merge<512, 2>), grid, dim3(512), 0, st, a);
    else if (per <= 8)
        hipLaunchKernelGGL((k_beam_merge<512, 8>), grid, dim3(512), 0, st, a);
    else
        hipLaunchKernelGGL((k_beam_merge<1024, 0>), grid, dim3(1024), 0, st, a);
    return hipGetLastError();
}

}  // namespace dhtop
