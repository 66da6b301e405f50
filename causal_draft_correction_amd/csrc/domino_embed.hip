// Embedding: rows of a table by token, scaled, and the gradient of the table.
//
//     out_i = scale table[id_i]                       (0 where id_i is outside [0, V))
//     dtable[v] = scale sum_{i: id_i = v} g_i         (in 32 bits, positions in ascending order; 0 where there are none)
//
// Both are bound by bytes.  The gradient sorts (token, position) pairs by token, stably, so that the positions of a
// token come one after the other; a block takes TILE sorted pairs and COLS columns, adds rows while the token stays
// the same, and writes the sum of each token whose pairs all lie in its tile.  A token that reaches over tiles (a
// frequent one, padding) leaves a partial sum in each, which k_embed_join adds in their order.  Nothing is added by
// atomics: the result does not change from call to call.
//
// Up to SORT_MAX tokens are sorted by one block, in LDS (6 bits a pass, ranks by ballots); the launch's other blocks
// meanwhile clear the table, which takes longer wherever the vocabulary is large.  Up to 256 tokens take one launch, whose
// blocks each look all tokens through for those of their rows; added to what is there, for the rows that are named alone.
//
// Measured on one MI355X.  Rows of 4096 bfloat16, 4096 tokens of 4096 rows (34 MB written, 23 read past the dies' caches):
// 8.6 to 11 us, 5 to 6.5 TB/s.  Gradient of 4096 tokens, 1024 float32, a table of 151936 rows: 95 us for sorting and 622 MB
// of zeros (6.6 TB/s, what a fill reaches), 8.5 us for the sums (16.8 MB, latency: 256 tiles, each with 8 rows in flight), 4.7
// for the join.  32 tokens of 64 over 1024 rows: 4.4 us, a call 8 us, sorted and joined 16.
#define DH_NT 256
#define DH_NS dhe
#include "dh_rows.h"
#include "dh_embed.h"

namespace DH_NS {

constexpr int DIGIT = 6, BINS = 1 << DIGIT;
constexpr int SORT_NT = 1024, SORT_NW = SORT_NT / 64;
constexpr int SORT_MAX = 8 * SORT_NT;  // pairs that one block sorts: 64 KiB
constexpr int SORT_TILE = 4 * SORT_NT;  // pairs a block takes where there are more
constexpr int COLS = 4 * NT;           // columns of a block of k_embed_sum

// A pair: its token (V where it names no row) and its position.
typedef uint2 Pair;

// Eight elements at any element address, as floats.
template <typename T>
__device__ inline void load8(const T *p, float (&f)[8])
{
    typedef Vec<T> VT;
#pragma unroll
    for (int u = 0; u < 8 / VT::N; ++u) {
        const typename VT::raw x = *reinterpret_cast<const typename VT::mem *>(p + u * VT::N);
#pragma unroll
        for (int e = 0; e < VT::N; ++e)
            f[u * VT::N + e] = VT::get(x, e);
    }
}
template <typename T>
__device__ inline void store8(T *p, const float (&f)[8])
{
    typedef Vec<T> VT;
#pragma unroll
    for (int u = 0; u < 8 / VT::N; ++u) {
        typename VT::raw x = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < VT::N; ++e)
            VT::set(x, e, f[u * VT::N + e]);
        *reinterpret_cast<typename VT::mem *>(p + u * VT::N) = x;
    }
}

// Part of a row: eight columns a thread, `per` threads a row.
template <typename TI, typename TO>
__global__ __launch_bounds__(NT) void k_embed(Rows table, const int32_t *ids, float scale, Rows out, uint32_t n,
                                              Divisor per)
{
    const uint32_t i = blockIdx.x * NT + threadIdx.x;  // (below 2^31: B R (V / 1024 + 1) is below 2^24)
    if (i >= n)
        return;
    const uint32_t row = per.quotient(i);
    const int c = static_cast<int>(i - row * per.d) * 8, d = table.V;
    const Place at = out.place(row);
    TO *o = const_cast<TO *>(row_at<TO>(out, at)) + c;
    const int id = ids[row];
    const bool in = id >= 0 && id < table.R;
    const TI *t = static_cast<const TI *>(table.data) + (in ? id : 0) * table.rs + c;
    if (c + 8 <= d) {
        float f[8] = {};
        if (in)
            load8(t, f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] *= in ? scale : 0.f;
        store8(o, f);
    } else {
        for (int e = 0; c + e < d; ++e)
            Vec<TO>::put(o + e, in ? scale * Vec<TI>::one(t + e) : 0.f);
    }
}

// ---- sorting ----

__device__ inline Pair pair_at(const int32_t *ids, int64_t n, int64_t i, int V)
{
    if (i >= n)
        return Pair{0xFFFFFFFFu, 0};
    const int id = ids[i];
    return Pair{id >= 0 && id < V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(V), static_cast<uint32_t>(i)};
}

// The place of the lane's digit among the equal ones of the wave's earlier calls and of lower lanes; `count`: the
// wave's numbers of each digit so far.
__device__ inline int wave_rank(uint32_t digit, volatile uint32_t *count)
{
    uint64_t same = ~0ull;
#pragma unroll
    for (int b = 0; b < DIGIT; ++b) {
        const uint64_t set = __ballot((digit >> b) & 1u);
        same &= (digit >> b) & 1u ? set : ~set;
    }
    const uint64_t below = same & ((1ull << (threadIdx.x & 63)) - 1);
    const uint32_t before = count[digit];
    __builtin_amdgcn_wave_barrier();
    if (!below)
        count[digit] = before + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    return static_cast<int>(before) + __popcll(below);
}

// Exclusive sum over the lanes.
__device__ inline uint32_t wave_before(uint32_t v)
{
    uint32_t sum = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t up = __shfl_up(sum, o);
        if ((threadIdx.x & 63) >= static_cast<unsigned>(o))
            sum += up;
    }
    return sum - v;
}

// Places of the block's E pairs a thread by one digit: those of wave w are its E * 64 neighbours, in the order of
// lanes, then of e.  place[e] counts from `base[digit]` (NULL: from the digit's place in the block).
template <int E>
__device__ inline void block_places(const Pair (&x)[E], int shift, uint32_t (&count)[SORT_NW][BINS],
                                    uint32_t (&start)[BINS], const uint32_t *base, uint32_t (&place)[E])
{
    const int wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < SORT_NW * BINS; i += SORT_NT)
        (&count[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e)
        place[e] = static_cast<uint32_t>(wave_rank((x[e].x >> shift) & (BINS - 1), count[wave]));
    __syncthreads();
    if (threadIdx.x < BINS) {
        uint32_t sum = 0;
        for (int w = 0; w < SORT_NW; ++w) {
            const uint32_t here = count[w][threadIdx.x];
            count[w][threadIdx.x] = sum;
            sum += here;
        }
        start[threadIdx.x] = base ? base[threadIdx.x] : wave_before(sum);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint32_t digit = (x[e].x >> shift) & (BINS - 1);
        place[e] += start[digit] + count[wave][digit];
    }
}

// Zeros for the rows of the table, by the blocks [0, blocks): in 16-byte stores where a row allows them.
template <typename T>
__device__ inline void clear_rows(const Rows &table, int64_t block, int64_t blocks, int threads)
{
    T *data = static_cast<T *>(const_cast<void *>(table.data));
    const int64_t step = blocks * threads, first = block * threads + threadIdx.x;
    if (table.rs == table.V) {  // one piece of memory: from its first address at 16 bytes on
        const int64_t n = static_cast<int64_t>(table.R) * table.V;
        const int64_t skew = (16 - reinterpret_cast<uintptr_t>(data) % 16) % 16 / sizeof(T);
        const int64_t head = skew < n ? skew : n, vecs = (n - head) / Vec<T>::N;
        typedef typename Vec<bf16s>::raw words;
        words *v = reinterpret_cast<words *>(data + head);
        // (a block's share in one piece: 622 MB in pieces of 16 KiB 95 us, strided over 512 blocks 122 us)
        const int64_t each = (vecs + blocks - 1) / blocks, from = block * each;
        for (int64_t i = from + threadIdx.x; i < from + each && i < vecs; i += threads)
            __builtin_nontemporal_store(words{0, 0, 0, 0}, v + i);
        const int64_t tail = head + vecs * Vec<T>::N;
        if (first < head)
            Vec<T>::put(data + first, 0.f);
        if (first < n - tail)
            Vec<T>::put(data + tail + first, 0.f);
    } else {
        const int per = (table.V + 7) / 8;
        const int64_t n = static_cast<int64_t>(table.R) * per;
        for (int64_t i = first; i < n; i += step) {
            const int64_t row = i / per;
            const int c = static_cast<int>(i - row * per) * 8;
            T *p = data + row * table.rs + c;
            if (c + 8 <= table.V) {
                const float zero[8] = {};
                store8(p, zero);
            } else {
                for (int e = 0; c + e < table.V; ++e)
                    Vec<T>::put(p + e, 0.f);
            }
        }
    }
}

// Block 0 sorts n <= E * SORT_NT tokens; the others clear the table.
template <typename T, int E>
__global__ __launch_bounds__(SORT_NT) void k_embed_sort(const int32_t *ids, int n, int V, int bits, Pair *sorted,
                                                        Rows table)
{
    __shared__ Pair list[E * SORT_NT];
    __shared__ uint32_t count[SORT_NW][BINS], start[BINS];
    if (blockIdx.x > 0) {
        clear_rows<T>(table, blockIdx.x - 1, gridDim.x - 1, SORT_NT);
        return;
    }
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, first = wave * E * 64 + lane;
    Pair x[E];
    uint32_t place[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        x[e] = pair_at(ids, n, first + e * 64, V);
    for (int shift = 0; shift < bits; shift += DIGIT) {
        block_places<E>(x, shift, count, start, nullptr, place);
#pragma unroll
        for (int e = 0; e < E; ++e)
            list[place[e]] = x[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[e] = list[first + e * 64];
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (first + e * 64 < n)
            sorted[first + e * 64] = x[e];
}

// One pass over more tokens: how many of each digit a block's tile has (hist[digit][block]); the first one's launch
// has blocks that clear the table, too.  `from`: the pairs in the order of the pass before, NULL in the first.
template <typename T>
__global__ __launch_bounds__(SORT_NT) void k_embed_hist(const int32_t *ids, const Pair *from, int64_t n, int V,
                                                        int shift, int tiles, uint32_t *hist, Rows table)
{
    __shared__ uint32_t count[BINS];
    if (static_cast<int>(blockIdx.x) >= tiles) {
        clear_rows<T>(table, blockIdx.x - tiles, gridDim.x - tiles, SORT_NT);
        return;
    }
    if (threadIdx.x < BINS)
        count[threadIdx.x] = 0;
    __syncthreads();
    for (int e = 0; e < SORT_TILE / SORT_NT; ++e) {
        const int64_t i = static_cast<int64_t>(blockIdx.x) * SORT_TILE + e * SORT_NT + threadIdx.x;
        if (i < n)
            atomicAdd(&count[((from ? from[i].x : pair_at(ids, n, i, V).x) >> shift) & (BINS - 1)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < BINS)
        hist[static_cast<int64_t>(threadIdx.x) * tiles + blockIdx.x] = count[threadIdx.x];
}

// Exclusive sums over hist[0, n), by one block.
__global__ __launch_bounds__(SORT_NT) void k_embed_scan(uint32_t *hist, int n)
{
    __shared__ uint32_t sums[SORT_NW];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    uint32_t before = 0;
    for (int i0 = 0; i0 < n; i0 += SORT_NT) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        const uint32_t v = i < n ? hist[i] : 0, ex = wave_before(v);
        if (lane == 63)
            sums[wave] = ex + v;
        __syncthreads();
        uint32_t here = before;
        for (int w = 0; w < SORT_NW; ++w) {
            here += w < wave ? sums[w] : 0;
            before += sums[w];
        }
        if (i < n)
            hist[i] = here + ex;
        __syncthreads();
    }
}

__global__ __launch_bounds__(SORT_NT) void k_embed_scatter(const int32_t *ids, const Pair *from, int64_t n, int V,
                                                           int shift, int tiles, const uint32_t *hist, Pair *to)
{
    constexpr int E = SORT_TILE / SORT_NT;
    __shared__ uint32_t count[SORT_NW][BINS], start[BINS], base[BINS];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * SORT_TILE + wave * E * 64 + lane;
    if (threadIdx.x < BINS)
        base[threadIdx.x] = hist[static_cast<int64_t>(threadIdx.x) * tiles + blockIdx.x];
    Pair x[E];
    uint32_t place[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int64_t i = first + e * 64;
        x[e] = i < n && from ? from[i] : pair_at(ids, n, i, V);
    }
    __syncthreads();
    // (pairs past the end have the largest digit and come last in the last tile: their places are past n)
    block_places<E>(x, shift, count, start, base, place);
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (first + e * 64 < n)
            to[place[e]] = x[e];
}

// ---- sums ----

// Four columns at any element address, those past `left` as zeros.
template <typename T>
__device__ inline void load4(const T *p, int left, float (&f)[4])
{
    if (left >= 4) {
        if constexpr (sizeof(T) == 4) {
            const typename Vec<T>::raw x = *reinterpret_cast<const typename Vec<T>::mem *>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = x[e];
        } else {
            typedef uint32_t two __attribute__((ext_vector_type(2), aligned(2)));
            const two x = *reinterpret_cast<const two *>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = __uint_as_float(e & 1 ? x[e >> 1] & 0xFFFF0000u : x[e >> 1] << 16);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f[e] = e < left ? Vec<T>::one(p + e) : 0.f;
    }
}
template <typename T>
__device__ inline void store4(T *p, int left, const float (&f)[4])
{
    if (left >= 4) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<typename Vec<T>::mem *>(p) = typename Vec<T>::raw{f[0], f[1], f[2], f[3]};
        } else {
            typedef uint32_t two __attribute__((ext_vector_type(2), aligned(2)));
            *reinterpret_cast<two *>(p) = two{Vec<T>::bits(f[0]) | (Vec<T>::bits(f[1]) << 16),
                                              Vec<T>::bits(f[2]) | (Vec<T>::bits(f[3]) << 16)};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left)
                Vec<T>::put(p + e, f[e]);
    }
}

// Four columns of a token's sum, scaled, to the table (or added to it).
template <typename T>
__device__ inline void put_sum(const Rows &table, uint32_t token, int c, float scale, bool accumulate,
                               const float (&sum)[4])
{
    T *p = static_cast<T *>(const_cast<void *>(table.data)) + static_cast<int64_t>(token) * table.rs + c;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (accumulate)
        load4(p, table.V - c, f);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        f[e] += scale * sum[e];
    store4(p, table.V - c, f);
}

struct Sums {
    const Pair *sorted;
    int64_t n;
    int tile;          // pairs of a tile
    int pitch;         // floats of a partial sum
    float *partial;    // [tiles, 2, pitch]: of the token that reaches into the tile from before it, or through it;
                       // of the one that begins in it and reaches past it
    float scale;
    bool accumulate;
};

template <typename TG, typename TT>
__global__ __launch_bounds__(NT) void k_embed_sum(Sums s, Rows grad, Rows table)
{
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * s.tile;
    const int64_t i1 = i0 + s.tile < s.n ? i0 + s.tile : s.n;
    const int c = static_cast<int>(blockIdx.y) * COLS + 4 * static_cast<int>(threadIdx.x), left = table.V - c;
    const uint32_t before = i0 ? s.sorted[i0 - 1].x : 0xFFFFFFFFu, after = i1 < s.n ? s.sorted[i1].x : 0xFFFFFFFFu;
    const uint32_t V = static_cast<uint32_t>(table.R);
    if (left <= 0)
        return;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t now = s.sorted[i0].x;
    auto flush = [&](bool last) {
        const bool from_before = now == before, past = last && now == after;
        if (now >= V)
            return;
        if (from_before || past) {
            float *p = s.partial + (2 * static_cast<int64_t>(blockIdx.x) + (from_before ? 0 : 1)) * s.pitch + c;
            store4(p, 4, sum);
        } else {
            put_sum<TT>(table, now, c, s.scale, s.accumulate, sum);
        }
    };
    constexpr int AHEAD = 8;  // rows in flight
    for (int64_t i = i0; i < i1; i += AHEAD) {
        Pair x[AHEAD];
        float f[AHEAD][4];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            x[u] = s.sorted[i + u < i1 ? i + u : i1 - 1];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            load4(row_at<TG>(grad, grad.place(x[u].y)) + c, left, f[u]);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (i + u < i1) {
                if (x[u].x != now) {
                    flush(false);
                    now = x[u].x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] += f[u][e];
            }
    }
    flush(true);
}

// A token that begins in tile blockIdx.x and reaches past it: the sum of its partial sums.  16 lanes take 64 columns,
// 16 groups of them every 16th tile.
template <typename TT>
__global__ __launch_bounds__(NT) void k_embed_join(Sums s, int tiles, Rows table)
{
    __shared__ float part[16][64];
    const int64_t end = (static_cast<int64_t>(blockIdx.x) + 1) * s.tile;  // (the last tile has no block)
    const uint32_t token = s.sorted[end - 1].x;
    if (token >= static_cast<uint32_t>(table.R) || s.sorted[end].x != token)
        return;
    const int64_t begin = end - s.tile;
    if (begin && s.sorted[begin - 1].x == token)
        return;  // (it began before)
    // the tiles that begin with the token follow one another
    int last = static_cast<int>(blockIdx.x);
    for (int more = NT; more == NT;) {
        const int64_t at = (static_cast<int64_t>(last) + 1 + threadIdx.x) * s.tile;
        more = __syncthreads_count(at < s.n && s.sorted[at].x == token);
        last += more;
    }
    const int group = threadIdx.x >> 4, c = static_cast<int>(blockIdx.y) * 64 + 4 * (static_cast<int>(threadIdx.x) & 15);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < s.pitch)
        for (int t = static_cast<int>(blockIdx.x) + group; t <= last; t += 16) {
            float f[4];
            load4(s.partial + (2 * static_cast<int64_t>(t) + (t == static_cast<int>(blockIdx.x))) * s.pitch + c, 4, f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[e] += f[e];
        }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        part[group][4 * (threadIdx.x & 15) + e] = sum[e];
    __syncthreads();
    if (group || c >= table.V)
        return;
    const int groups = last - static_cast<int>(blockIdx.x) + 1 < 16 ? last - static_cast<int>(blockIdx.x) + 1 : 16;
    for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum[e] += part[g][4 * (threadIdx.x & 15) + e];
    put_sum<TT>(table, token, c, s.scale, s.accumulate, sum);
}

// ---- few tokens ----

// The places of the block's hits in their order (thread after thread); returns how many there are.  Two barriers.
__device__ inline int ordered_places(bool hit, uint32_t *count, int &place)
{
    const int wave = threadIdx.x >> 6;
    const uint64_t mask = __ballot(hit);
    if ((threadIdx.x & 63) == 0)
        count[wave] = __popcll(mask);
    __syncthreads();
    place = __popcll(mask & ((1ull << (threadIdx.x & 63)) - 1));
    int all = 0;
#pragma unroll
    for (int w = 0; w < NWAVE; ++w) {
        place += w < wave ? static_cast<int>(count[w]) : 0;
        all += static_cast<int>(count[w]);
    }
    __syncthreads();
    return all;
}

// At most NT tokens, one a thread: a block writes `per` rows of the table, those of its tokens and zeros for the others;
// with `accumulate` (per = 1) a block for each place, of which a token's first has its row, and for every 4 NT columns.
template <typename TG, typename TT>
__global__ __launch_bounds__(NT) void k_embed_few(const int32_t *ids, int n, float scale, bool accumulate, int per,
                                                  Rows grad, Rows table)
{
    __shared__ int token[NT], at[NT], mine[NT];
    __shared__ uint32_t count[NWAVE];
    __shared__ uint8_t named[NT];
    const int64_t row0 = accumulate ? ids[blockIdx.x] : static_cast<int64_t>(blockIdx.x) * per;
    const int64_t row1 = row0 + per < table.R ? row0 + per : table.R;
    if (row0 < 0 || row0 >= table.R)
        return;
    const int t = threadIdx.x, id = t < n ? ids[t] : -1;
    const bool hit = id >= row0 && id < row1;
    int place;
    named[t] = 0;
    const int hits = ordered_places(hit, count, place);
    if (hit) {
        token[place] = id;
        at[place] = t;
        named[id - row0] = 1;
    }
    __syncthreads();
    if (accumulate && at[0] != static_cast<int>(blockIdx.x))
        return;
    const int d = table.V, quads = (d + 3) / 4, rows = static_cast<int>(row1 - row0);
    TT *out = static_cast<TT *>(const_cast<void *>(table.data)) + row0 * table.rs;
    if (!accumulate)
        for (int i = t; i < rows * quads; i += NT) {
            const int r = i / quads, c = 4 * (i - r * quads);
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            if (!named[r])
                store4(out + r * table.rs + c, d - c, zero);
        }
    for (int h = 0; h < hits; ++h) {
        const int now = token[h];
        if (!named[now - row0])
            continue;  // (an earlier place took them all)
        const bool same = t < hits && token[t] == now;
        const int all = ordered_places(same, count, place);
        if (same)
            mine[place] = at[t];
        if (t == 0)
            named[now - row0] = 0;
        __syncthreads();
        for (int c = 4 * (t + NT * static_cast<int>(blockIdx.y)); c < d; c += 4 * NT * static_cast<int>(gridDim.y)) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            constexpr int AHEAD = 8;
            for (int i = 0; i < all; i += AHEAD) {
                float f[AHEAD][4];
#pragma unroll
                for (int u = 0; u < AHEAD; ++u)
                    load4(row_at<TG>(grad, grad.place(mine[i + u < all ? i + u : all - 1])) + c, d - c, f[u]);
#pragma unroll
                for (int u = 0; u < AHEAD; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[e] += i + u < all ? f[u][e] : 0.f;
            }
            put_sum<TT>(table, now, c, scale, accumulate, sum);
        }
        __syncthreads();
    }
}

}  // namespace DH_NS

namespace dhembed {

using namespace dhe;

namespace {

template <typename F>
void by_type(int dtype, F f)
{
    if (dtype == DOMINO_F32)
        f(float{});
    else
        f(bf16s{});
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

struct Layout {
    int64_t n;
    int tile, tiles, sort_tiles, pitch;
    size_t sorted, other, hist, partial, bytes;
};

// Tiles of 16 pairs, so that few tokens still give blocks for every compute unit; of 64 where they are many.
Layout layout_of(const domino_rows &grad)
{
    Layout l;
    l.n = static_cast<int64_t>(grad.B) * grad.R;
    l.tile = l.n > 16 * 1024 ? 64 : 16;
    l.tiles = static_cast<int>((l.n + l.tile - 1) / l.tile);
    l.sort_tiles = l.n > SORT_MAX ? static_cast<int>((l.n + SORT_TILE - 1) / SORT_TILE) : 0;
    l.pitch = (grad.V + 3) / 4 * 4;
    size_t at = 0;
    l.sorted = at, at += round16(l.n * sizeof(Pair));
    l.other = at, at += l.sort_tiles ? round16(l.n * sizeof(Pair)) : 0;
    l.hist = at, at += round16(static_cast<size_t>(l.sort_tiles) * BINS * sizeof(uint32_t));
    l.partial = at, at += static_cast<size_t>(l.tiles) * 2 * l.pitch * sizeof(float);
    l.bytes = at;
    return l;
}

}  // namespace

hipError_t forward(const domino_rows &table, const int32_t *ids, float scale, const domino_rows &out, hipStream_t st)
{
    const int per = (table.V + 7) / 8;
    const int64_t n = static_cast<int64_t>(out.B) * out.R * per;
    const Rows t = rows_of(table, nullptr, false), o = rows_of(out, nullptr, false);
    const dim3 grid(static_cast<unsigned>((n + NT - 1) / NT));
    by_type(table.dtype, [&](auto in) {
        by_type(out.dtype, [&](auto to) {
            hipLaunchKernelGGL((k_embed<decltype(in), decltype(to)>), grid, dim3(NT), 0, st, t, ids, scale, o,
                               static_cast<uint32_t>(n), divisor(static_cast<uint32_t>(per)));
        });
    });
    return hipGetLastError();
}

// Tokens that one launch takes, each block with its own rows of the table: no more than that many gradients are added in
// turn, and every block reads them all.  (A token repeated takes its block longer: of 1024 float32 columns and 151936 rows,
// 256 tokens 108 us, all of them the same 156, and 257, sorted, 100 either way; added to what is there, 7, 63 and 15.)
constexpr int FEW = NT;

size_t workspace_bytes(const domino_rows &grad)
{
    return static_cast<int64_t>(grad.B) * grad.R <= FEW ? 0 : layout_of(grad).bytes;
}

hipError_t backward(const domino_rows &grad, const int32_t *ids, float scale, bool accumulate, void *ws,
                    const domino_rows &table, hipStream_t st)
{
    if (static_cast<int64_t>(grad.B) * grad.R <= FEW) {
        // 16 KiB of the table a block, and no more than makes 512 blocks: a block takes its tokens one after the other.  Added
        // to what is there, other rows are of no account: a block a place (32 tokens of 4096 float32 columns, a table of
        // 151936 rows: 40 us with blocks for all rows, 7 so).
        const int n = grad.B * grad.R;
        const int64_t row = static_cast<int64_t>(table.V) * (table.dtype == DOMINO_F32 ? 4 : 2);
        int64_t per = 16384 / row < table.R / 512 ? 16384 / row : table.R / 512;
        per = per < 1 || accumulate ? 1 : per > NT ? NT : per;
        const dim3 grid = accumulate ? dim3(n, static_cast<unsigned>((table.V + 4 * NT - 1) / (4 * NT)))
                                     : dim3(static_cast<unsigned>((table.R + per - 1) / per));
        const Rows g = rows_of(grad, nullptr, false), t = rows_of(table, nullptr, false);
        by_type(table.dtype, [&](auto to) {
            by_type(grad.dtype, [&](auto from) {
                hipLaunchKernelGGL((k_embed_few<decltype(from), decltype(to)>), grid, dim3(NT), 0, st, ids, n, scale,
                                   accumulate, static_cast<int>(per), g, t);
            });
        });
        return hipGetLastError();
    }
    const Layout l = layout_of(grad);
    char *base = static_cast<char *>(ws);
    Pair *sorted = reinterpret_cast<Pair *>(base + l.sorted), *other = reinterpret_cast<Pair *>(base + l.other);
    uint32_t *hist = reinterpret_cast<uint32_t *>(base + l.hist);
    const Rows g = rows_of(grad, nullptr, false), t = rows_of(table, nullptr, false);
    const int V = table.R;
    int bits = 1;
    while (bits < 31 && (V >> bits))
        ++bits;  // V itself stands for no row
    // blocks that clear the table: one store a thread
    const int64_t size = static_cast<int64_t>(table.R) * table.V * (table.dtype == DOMINO_F32 ? 4 : 2);
    const int64_t want = (size + 16 * SORT_NT - 1) / (16 * SORT_NT);
    const unsigned clears = accumulate ? 0 : static_cast<unsigned>(want < 1 << 20 ? want : 1 << 20);
    hipError_t e;
    if (!l.sort_tiles) {
        const int n = static_cast<int>(l.n);
        by_type(table.dtype, [&](auto to) {
            typedef decltype(to) T;
            const dim3 grid(1 + clears), block(SORT_NT);
            if (n <= SORT_NT)
                hipLaunchKernelGGL((k_embed_sort<T, 1>), grid, block, 0, st, ids, n, V, bits, sorted, t);
            else if (n <= 4 * SORT_NT)
                hipLaunchKernelGGL((k_embed_sort<T, 4>), grid, block, 0, st, ids, n, V, bits, sorted, t);
            else
                hipLaunchKernelGGL((k_embed_sort<T, 8>), grid, block, 0, st, ids, n, V, bits, sorted, t);
        });
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    } else {
        const int passes = (bits + DIGIT - 1) / DIGIT;
        const Pair *from = nullptr;
        for (int p = 0; p < passes; ++p) {
            Pair *to = (passes - 1 - p) & 1 ? other : sorted;
            const unsigned extra = p ? 0 : clears;
            by_type(table.dtype, [&](auto type) {
                hipLaunchKernelGGL((k_embed_hist<decltype(type)>), dim3(l.sort_tiles + extra), dim3(SORT_NT), 0, st,
                                   ids, from, l.n, V, p * DIGIT, l.sort_tiles, hist, t);
            });
            if ((e = hipGetLastError()) != hipSuccess)
                return e;
            hipLaunchKernelGGL(k_embed_scan, dim3(1), dim3(SORT_NT), 0, st, hist, l.sort_tiles * BINS);
            hipLaunchKernelGGL(k_embed_scatter, dim3(l.sort_tiles), dim3(SORT_NT), 0, st, ids, from, l.n, V,
                               p * DIGIT, l.sort_tiles, hist, to);
            if ((e = hipGetLastError()) != hipSuccess)
                return e;
            from = to;
        }
    }
    const Sums s = {sorted, l.n, l.tile, l.pitch, reinterpret_cast<float *>(base + l.partial), scale, accumulate};
    by_type(table.dtype, [&](auto to) {
        by_type(grad.dtype, [&](auto from) {
            hipLaunchKernelGGL((k_embed_sum<decltype(from), decltype(to)>),
                               dim3(l.tiles, static_cast<unsigned>((grad.V + COLS - 1) / COLS)), dim3(NT), 0, st, s, g,
                               t);
        });
        if (l.tiles > 1)
            hipLaunchKernelGGL((k_embed_join<decltype(to)>),
                               dim3(l.tiles - 1, static_cast<unsigned>((grad.V + 63) / 64)), dim3(NT), 0, st, s,
                               l.tiles, t);
    });
    return hipGetLastError();
}

}  // namespace dhembed
