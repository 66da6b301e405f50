// Distillation of the head from a teacher's top logits: the loss of a student's rows, and its gradient.
//
// With y = z / tau, q = softmax(y), the teacher's entries j (id in [0, V)), t_j = value_j / tau - L with L the
// teacher's log-sum-exp (given, or that of the entries alone), p_j = exp t_j, P = sum p_j,
//     rest = max(0, 1 - P) where L is given, else 0;   Mm = P + rest;   Qr = sum of q over ids no entry names
//     (where 1 - P is no more than the rounding of L leaves open, and Qr than the square of that: as if L were not given)
//     loss = tau^2 [ sum_j p_j (t_j - log q_j) + rest log(rest / Qr) ]
//     dloss/dz_v = tau [ Mm q_v - sum_{j: id_j = v} p_j ]     where an entry names v
//                = tau (q_v / Qr) [ Mm Qr - rest ]             elsewhere
// The sum over the ids that no entry names is taken by itself (named elements count as -inf), never as a
// difference, and has a maximum of its own; the named elements are added in 64 bits.  So log s and Qr both keep their
// precision where the student is nearly certain of a named id and the loss is small.
//
// The forward pass reads a row once (k_distill_part, one block per chunk, values in registers) and joins the
// chunks and the k entries in 64 bits (k_distill_final).  The backward pass reads it once and writes it once
// (k_distill_grad).  Rows that one block can hold go through one launch (k_distill_row): 32 f32 rows of 1024, loss and
// gradient: 6.8 us, against 3.4 + 6.2 + 3.0 us and two more launches.
//
// What bounds them, on one MI355X.  1024 f32 rows of 151936 (622 MB), loss and gradient: 92 + 8.3 + 196 us, 6.8 TB/s
// read, then 6.4 TB/s read and written; a large copy reaches 4.9 TB/s.  512 bf16 rows (156 MB): 29 + 5.5 + 46 us; in
// bfloat16 the forward pass is bound by the vector units (552 instructions a wave, 59 of them exponentials: 24 us of
// issue) as much as by the bytes (24 us).  The gradient needs the row's sum, so a row is read twice, from HBM where
// the last-level cache does not hold it.  Keeping a row on chip between the two passes, one block of 256 to 1024
// threads per row that reads its tiles again in the opposite order, was measured at 303 to 314 us for the f32 rows
// and 164 to 189 us for 1024 bf16 ones (three launches: 294 and 159 us): a block's passes wait for each other.
// k_distill_grad takes 4 vectors a thread: 194 us against 200 us with 8 and 198 us with 2; k_distill_part 8: in bf16
// 26.6 us against 28.4 us with 4.
#define DH_NT 256
#define DH_NS dhd
#include "dh_rows.h"
#include "dh_distill.h"

namespace DH_NS {

constexpr int MAX_IDS = dhdistill::MAX_K, HEAD = dhdistill::STAT_HEAD;
static_assert(MAX_IDS == 128 && MAX_IDS <= NT, "one thread, or half a lane, per id");

struct Teach {
    int k;
    const int32_t *ids;
    const float *values, *lse;
};

__device__ inline bool in_row(int id, int V) { return id >= 0 && id < V; }

// One bit for each element of a chunk that an entry names, in the words of the thread that holds it.
template <typename T, int NV>
constexpr int MASK_WORDS = (NV * Vec<T>::N + 31) / 32;

template <int WORDS, int NTB>
__device__ inline void clear_mask(uint32_t (&mask)[WORDS][NTB])
{
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
        mask[i][threadIdx.x] = 0;
}

// Named elements of the chunk [v0, v1) become -inf.  `id`: the thread's entry, or -1.  The mask was cleared before
// the block's last barrier.
template <typename T, int NV, int WORDS, int NTB>
__device__ inline void drop_named(typename Vec<T>::raw (&x)[NV], uint32_t (&mask)[WORDS][NTB], int id, int v0, int v1)
{
    typedef Vec<T> VT;
    if (id >= v0 && id < v1) {
        const int o = id - v0, i = o / VT::N, bit = i / NTB * VT::N + o % VT::N;
        atomicOr(&mask[bit >> 5][i % NTB], 1u << (bit & 31));
    }
    __syncthreads();
    uint32_t mine[WORDS], any = 0;
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
        any |= mine[i] = mask[i][threadIdx.x];
    if (any) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const uint32_t bits = (mine[u * VT::N >> 5] >> (u * VT::N & 31)) & ((1u << VT::N) - 1);
            if (bits) {
#pragma unroll
                for (int e = 0; e < VT::N; ++e)
                    if ((bits >> e) & 1u)
                        VT::set(x[u], e, NEG_INF);
            }
        }
    }
}

// The block's maximum and sum of exponentials (a NaN or +inf makes both NaN: so the row's), in every thread.
template <typename T, int NV, int NTB>
__device__ inline Part chunk_part(typename Vec<T>::raw (&x)[NV], const Scale &sc, float *red_m, float *red_s)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    float m = NEG_INF;
#pragma unroll
    for (int u = 0; u < NV; ++u)
        m = Vec<T>::max_with(x[u], m);
    m = wave_max(m);
    if (lane == 0)
        red_m[wave] = m;
    __syncthreads();
    m = red_m[0];
#pragma unroll
    for (int w = 1; w < NTB / 64; ++w)
        m = fmaxf(m, red_m[w]);
    const Expo ex(m > NEG_INF ? m : 0.f, sc);
    float s = ex.small ? sum_exps<T, true>(x, ex, sc) : sum_exps<T, false>(x, ex, sc);
    s = wave_sum(s);
    if (lane == 0)
        red_s[wave] = s;
    __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < NTB / 64; ++w)
        total += static_cast<double>(red_s[w]);
    total *= ex.fix(sc);
    return Part{total != total ? __builtin_nanf("") : m, total};
}

// The chunk's part, over the elements that no entry names.
template <typename T, int NV>
__global__ __launch_bounds__(NT) void k_distill_part(Rows rows, Teach te, Split sp, bool keep, Scale sc, Part *parts)
{
    __shared__ uint32_t mask[MASK_WORDS<T, NV>][NT];
    __shared__ float red_m[NWAVE], red_s[NWAVE];
    const int i_row = static_cast<int>(sp.by.quotient(blockIdx.x)), c = static_cast<int>(blockIdx.x) - i_row * sp.nch;
    const Place place = rows.place(i_row);
    const int row = place.row, cvec = sp.cvec;
    if (!rows.counts(place.b, place.r))
        return;
    int id = -1;
    if (static_cast<int>(threadIdx.x) < te.k)
        id = te.ids[static_cast<int64_t>(row) * te.k + threadIdx.x];
    clear_mask(mask);
    if (!__syncthreads_or(in_row(id, rows.V)))
        return;
    typename Vec<T>::raw x[NV];
    const T *z = row_at<T>(rows, place);
    if (keep)
        load_chunk<T, NV, NT, true>(x, z, rows.V, c, cvec);
    else
        load_chunk<T, NV>(x, z, rows.V, c, cvec);
    drop_named<T, NV>(x, mask, id, chunk_begin<T>(c, cvec, rows.V), chunk_begin<T>(c + 1, cvec, rows.V));
    const Part part = chunk_part<T, NV, NT>(x, sc, red_m, red_s);
    if (threadIdx.x == 0)
        parts[static_cast<int64_t>(row) * sp.nch + c] = part;
}

// L is a float32, so the masses p_j carry its rounding, up to |L| 2^-24, and the error of the sum it was taken from
// (LSE_STEPS half steps: an exponential's own 2, its argument's, 15 of a thread's additions).  Where 1 - sum p is no more
// than that noise, rest log(rest / Qr) is at most noise log(1 / noise) while Qr exceeds noise^2; below, it would be as
// large as Qr is small, up to an infinity (entries that name every id, or a mask that both share), made of nothing.
// An L so large that the noise exceeds MAX_NOISE tells nothing of the other ids (a row at the type's lowest value, whose L
// is -inf in float32 at temperatures below 1): such a row counts as given without it.
constexpr double LSE_STEPS = 32.0, MAX_NOISE = 0x1p-6;

// One row, by one wave, from the parts of its nch chunks: its loss, and what the backward pass needs of it:
//     stats = { m of the other ids, A, 1 (0: a row that is left out), log-sum-exp, h_0 .. h_{k-1} }
// so that dloss/dz_v = tau A exp((z_v - m) / tau), and tau h_j for v = id_j.  A lane takes the entries lane and
// lane + 64.  Everything is in 64 bits; differences are taken from the maxima, before their logarithms: rows at the
// type's lowest value keep them.
template <typename T>
__device__ inline void finish_row(const Rows &rows, const Teach &te, const Place &place, int nch, double tau,
                                  const Part *parts, float *loss, float *st, int *s_id, double *s_p)
{
    const double NINF = -__builtin_huge_val();
    const int lane = threadIdx.x & 63;
    const double inv_tau = 1.0 / tau;
    const int row = place.row;
    const int64_t at = static_cast<int64_t>(row) * te.k;
    const T *zr = row_at<T>(rows, place);
    const Part part = first_part(parts, nch);
    int id[2] = {-1, -1};
    float value[2] = {NEG_INF, NEG_INF};
    const double L = te.lse ? static_cast<double>(te.lse[row]) : NINF;
    const double noise = (fabs(L) + LSE_STEPS) * 0x1p-24;
    const bool told = te.lse && !(noise > MAX_NOISE && L < -NINF);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 64 * i < te.k) {
            id[i] = te.ids[at + lane + 64 * i];
            value[i] = te.values[at + lane + 64 * i];
        }
    if (!rows.counts(place.b, place.r))
        id[0] = id[1] = -1;
    double t[2] = {NINF, NINF}, z[2] = {NINF, NINF};
    bool valid[2];
    int own[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        valid[i] = in_row(id[i], rows.V);
        if (valid[i]) {
            t[i] = static_cast<double>(value[i]) * inv_tau;
            z[i] = Vec<T>::one(zr + id[i]);
        }
        own[i] = valid[i] ? id[i] : -1 - (lane + 64 * i);  // (invalid ones differ from all others)
        s_id[lane + 64 * i] = own[i];
    }
    // t becomes the logarithm of an entry's mass (without L: of its mass times p_sum)
    bool live = __ballot(valid[0] || valid[1]) != 0;
    double p[2] = {0.0, 0.0};
    double t_top = live ? wave_max_f64(fmax(t[0], t[1])) : NINF;
    if (live && !told && !(t_top > NINF)) {  // nothing but -inf (no mass: left out) or NaN
        live = __ballot((valid[0] && t[0] != t[0]) || (valid[1] && t[1] != t[1])) != 0;
        t_top = __builtin_nan("");
    }
    if (told)
        t_top = L;
    if (!live) {
        if (lane == 0)
            loss[row] = 0.f;
        if (st)
            for (int i = lane; i < HEAD + te.k; i += 64)
                st[i] = 0.f;
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (valid[i]) {
            t[i] -= t_top;
            p[i] = exp(t[i]);
        }
    const double p_sum = wave_sum_f64(p[0] + p[1]);
    float m_rest;
    double s_rest;
    join_parts(part, parts, nch, inv_tau, m_rest, s_rest);
    // entries that name an id again: the first of them stands for it, with the mass of all
    double named[2] = {p[0], p[1]};
    bool first[2] = {valid[0], valid[1]};
    s_p[lane] = p[0], s_p[lane + 64] = p[1];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    // entries with the lane's ids: one each, the entry itself, where no id is named twice
    int same[2] = {0, 0};
    const int4 *four = reinterpret_cast<const int4 *>(s_id);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int4 o = four[j];
        same[0] += (o.x == own[0]) + (o.y == own[0]) + (o.z == own[0]) + (o.w == own[0]);
    }
    if (te.k > 64) {
#pragma unroll 4
        for (int j = 0; j < 32; ++j) {
            const int4 o = four[j];
            same[1] += (o.x == own[1]) + (o.y == own[1]) + (o.z == own[1]) + (o.w == own[1]);
            if (j >= 16)
                same[0] += (o.x == own[0]) + (o.y == own[0]) + (o.z == own[0]) + (o.w == own[0]);
        }
    }
    if (__ballot(same[0] > 1 || same[1] > 1)) {
        named[0] = named[1] = 0.0;
        for (int j = 0; j < te.k; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (valid[i] && s_id[j] == id[i]) {
                    named[i] += s_p[j];
                    first[i] = first[i] && j >= lane + 64 * i;
                }
    }
    // the student's maximum; its sum over the other ids, and over all: the named ones, one by one, are in 64 bits, so
    // that log s keeps its digits where they have nearly all of the mass
    const double top = wave_max_f64(fmax(z[0], z[1]));
    const double m = m_rest > top || m_rest != m_rest ? m_rest : top;
    const double of_rest =
        m_rest == NEG_INF ? 0.0 : m_rest == m ? s_rest : s_rest * exp((m_rest - m) * inv_tau);
    double q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        q[i] = !valid[i] || m == NINF ? 0.0 : z[i] == m ? 1.0 : exp((z[i] - m) * inv_tau);
    const double s = wave_sum_f64((first[0] ? q[0] : 0.0) + (first[1] ? q[1] : 0.0)) + of_rest;
    bool alone = !told;  // the entries are all of the teacher: their masses are brought to a sum of 1
    double rest = 0.0;
    if (told) {
        rest = 1.0 - p_sum;
        alone = noise <= MAX_NOISE && fabs(rest) <= noise && of_rest <= noise * noise * s;
        rest = alone || rest < 0.0 ? 0.0 : rest;
    }
    const double scale = alone ? 1.0 / p_sum : 1.0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        p[i] *= scale, named[i] *= scale;
    // four logarithms, one in each of the first lanes
    const double logs = log(lane == 0 ? s : lane == 1 ? s_rest : lane == 2 ? rest : p_sum);
    const double log_s = __shfl(logs, 0), log_s_rest = __shfl(logs, 1), log_r = __shfl(logs, 2);
    const double log_p = alone ? __shfl(logs, 3) : 0.0;
    const double total = p_sum * scale + rest;
    const double lse = m == NINF ? NINF : m * inv_tau + log_s;
    double terms = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double logq = z[i] == NINF ? NINF : (z[i] - m) * inv_tau - log_s;
        terms += p[i] == 0.0 ? 0.0 : p[i] * ((t[i] - log_p) - logq);
    }
    double sum = wave_sum_f64(terms);
    const double inv_s = s > 0.0 || s != s ? 1.0 / s : 0.0;
    if (rest > 0.0)
        sum += rest * (log_r - (m_rest == NEG_INF ? NINF : (m_rest - m) * inv_tau + log_s_rest - log_s));
    double A = m_rest == NEG_INF ? 0.0 : (total * of_rest * inv_s - rest) / s_rest;
    const bool none = !(lse < -NINF);  // a NaN or +inf among the logits: no distribution
    if (none)
        sum = A = __builtin_nan("");
    if (lane == 0)
        loss[row] = static_cast<float>(tau * tau * sum);
    if (st) {
        if (lane == 0) {
            st[0] = m_rest > NEG_INF || m_rest != m_rest ? m_rest : 0.f;
            st[1] = static_cast<float>(A);
            st[2] = 1.f;
            st[3] = static_cast<float>(lse);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 64 * i < te.k)
                st[HEAD + lane + 64 * i] =
                    none ? __builtin_nanf("") : static_cast<float>(total * q[i] * inv_s - named[i]);
    }
}

template <typename T>
__global__ __launch_bounds__(NT) void k_distill_final(Rows rows, Teach te, int n_all, int nch, double tau,
                                                      const Part *parts, float *loss, float *stats)
{
    __shared__ __align__(16) int s_id[NWAVE][MAX_IDS];
    __shared__ double s_p[NWAVE][MAX_IDS];
    const int wave = threadIdx.x >> 6, i = blockIdx.x * NWAVE + wave;
    if (i >= n_all)
        return;
    const Place place = rows.place(i);
    finish_row<T>(rows, te, place, nch, tau, parts + static_cast<int64_t>(place.row) * nch, loss,
                  stats ? stats + static_cast<int64_t>(place.row) * (HEAD + te.k) : nullptr, s_id[wave], s_p[wave]);
}

// The chunk's elements become A exp((z - m) / tau), or 0 in rows left out.
template <typename T, int NV>
__device__ inline void chunk_grad(typename Vec<T>::raw (&x)[NV], bool live, float m, float A, const Scale &sc)
{
    if (!live) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            x[u] = typename Vec<T>::raw{0, 0, 0, 0};
        return;
    }
    const Expo ex(m, sc);
    const float a = A * static_cast<float>(ex.fix(sc));
    if (ex.small) {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            Vec<T>::map(x[u], [&](float z) { return a * ex.at<true>(z, sc); });
    } else {
#pragma unroll
        for (int u = 0; u < NV; ++u)
            Vec<T>::map(x[u], [&](float z) { return a * ex.at<false>(z, sc); });
    }
}

// dloss/dz of one chunk.  The elements that entries name are written again once the block's other stores are done.
template <typename T, int NV>
__global__ __launch_bounds__(NT) void k_distill_grad(Rows rows, int k, Split sp, const int32_t *ids,
                                                     const float *stats, const float *grad_loss, float tau, Scale sc,
                                                     Rows grad)
{
    const int i_row = static_cast<int>(sp.by.quotient(blockIdx.x)), c = static_cast<int>(blockIdx.x) - i_row * sp.nch;
    const Place place = rows.place(i_row);
    const int row = place.row, cvec = sp.cvec;
    T *out = const_cast<T *>(row_at<T>(grad, place));
    const float *st = stats + static_cast<int64_t>(row) * (HEAD + k);
    const bool counts = rows.counts(place.b, place.r);
    const int v0 = chunk_begin<T>(c, cvec, rows.V), v1 = chunk_begin<T>(c + 1, cvec, rows.V);
    typename Vec<T>::raw x[NV];
    if (counts)
        load_chunk<T, NV>(x, row_at<T>(rows, place), rows.V, c, cvec);
    const bool live = counts && st[2] != 0.f;
    const float g = grad_loss[row] * tau;
    chunk_grad<T, NV>(x, live, st[0], st[1] * g, sc);
    store_chunk<T, NV>(x, out, v0, v1);
    if (!live)
        return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the block's stores are done
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < k) {
        const int id = ids[static_cast<int64_t>(row) * k + threadIdx.x];
        if (id >= v0 && id < v1)
            Vec<T>::put(out + id, st[HEAD + threadIdx.x] * g);
    }
}

// A row of at most NV vectors a thread, by one block: loss, and with GRAD its gradient (else the statistics for a
// later backward pass).  The row stays in registers from its maximum to its gradient: it is read once.
template <typename T, int NTB, int NV, bool GRAD>
__global__ __launch_bounds__(NTB) void k_distill_row(Rows rows, Teach te, double tau, Scale sc, float *loss,
                                                    float *stats, const float *grad_loss, Rows grad)
{
    typedef Vec<T> VT;
    __shared__ float red_m[NTB / 64], red_s[NTB / 64];
    __shared__ Part part;
    __shared__ uint32_t mask[MASK_WORDS<T, NV>][NTB];
    __shared__ __align__(16) int s_id[MAX_IDS];
    __shared__ double s_p[MAX_IDS];
    __shared__ float s_stat[HEAD + MAX_IDS];
    const Place place = rows.place(blockIdx.x);
    const int row = place.row;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int id = -1;
    if (static_cast<int>(threadIdx.x) < te.k && rows.counts(place.b, place.r))
        id = te.ids[static_cast<int64_t>(row) * te.k + threadIdx.x];
    clear_mask(mask);
    typename VT::raw x[NV];
    const bool any = __syncthreads_or(in_row(id, rows.V));
    if (any) {
        load_chunk<T, NV, NTB>(x, row_at<T>(rows, place), rows.V, 0, NV * NTB);
        drop_named<T, NV>(x, mask, id, 0, rows.V);  // (their gradients are written last)
        const Part got = chunk_part<T, NV, NTB>(x, sc, red_m, red_s);
        if (threadIdx.x == 0)
            part = got;
    }
    __syncthreads();
    if (wave == 0) {
        if (any) {
            finish_row<T>(rows, te, place, 1, tau, &part, loss, s_stat, s_id, s_p);
        } else {
            for (int i = lane; i < HEAD + te.k; i += 64)
                s_stat[i] = 0.f;
            if (lane == 0)
                loss[row] = 0.f;
        }
    }
    __syncthreads();
    if constexpr (GRAD) {
        T *out = const_cast<T *>(row_at<T>(grad, place));
        const float g = grad_loss[row] * static_cast<float>(tau);
        const bool live = s_stat[2] != 0.f;
        chunk_grad<T, NV>(x, live, s_stat[0], s_stat[1] * g, sc);
        store_chunk<T, NV, NTB>(x, out, 0, rows.V);
        if (live) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the block's stores are done
            __syncthreads();
            if (in_row(id, rows.V))
                VT::put(out + id, s_stat[HEAD + threadIdx.x] * g);
        }
    } else if (stats) {
        for (int i = threadIdx.x; i < HEAD + te.k; i += NTB)
            stats[static_cast<int64_t>(row) * (HEAD + te.k) + i] = s_stat[i];
    }
}

}  // namespace DH_NS

namespace dhdistill {

using namespace dhd;

namespace {

constexpr int TARGET_BLOCKS = 1024;
constexpr int PART_NV = 8;        // vectors a thread takes at most: forward
constexpr int GRAD_NV = 4;    // backward

int vectors(const domino_logits &lg)
{
    const int per = lg.dtype == DOMINO_F32 ? 4 : 8;
    return static_cast<int>((static_cast<int64_t>(lg.V) + per - 1) / per);
}

// Rows that one block takes whole: up to 8 vectors for each of 1024 threads.  For the gradient always (read once
// instead of twice): 16, 256 and 1024 f32 rows of 32000 in 12.7, 17.6 and 66.0 us a call, in three launches 17.8, 25.5
// and 70.5 us; 1024 bf16 rows of 64000 72.7 and 72.0 us.  For the loss alone, where blocks of more than 512 threads
// would wait for each other's phases, up to one row a compute unit: 256 and 1024 f32 rows of 32000 in 12.8 and 42.5
// us, in two launches 15.9 and 30.5 us.
bool whole_rows(const domino_logits &lg, bool grad)
{
    const int nvec = vectors(lg);
    return nvec <= 512 * 8 || (nvec <= 1024 * 8 && (grad || static_cast<int64_t>(lg.B) * lg.R <= 256));
}

Split split_of(const domino_logits &lg, int max_nv)
{
    const int64_t rows = static_cast<int64_t>(lg.B) * lg.R;
    const int nvec = vectors(lg);
    const int least = static_cast<int>((static_cast<int64_t>(nvec) + NT * max_nv - 1) / (NT * max_nv));
    int64_t n = rows ? (TARGET_BLOCKS + rows - 1) / rows : 1;
    n = n < nvec / NT ? n : nvec / NT;
    n = n > least ? n : least;
    return split(nvec, n);
}

struct PartCall {
    bool keep;
    Rows rows;
    Teach te;
    Split sp;
    Scale sc;
    Part *parts;
    unsigned grid;
    hipStream_t st;
    template <typename T, int NV>
    void run() const
    {
        hipLaunchKernelGGL((k_distill_part<T, NV>), dim3(grid), dim3(NT), 0, st, rows, te, sp, keep, sc, parts);
    }
};

struct GradCall {
    Rows rows, grad;
    int k;
    const int32_t *ids;
    const float *stats, *grad_loss;
    double tau;
    Split sp;
    Scale sc;
    unsigned grid;
    hipStream_t st;
    template <typename T, int NV>
    void run() const
    {
        if constexpr (NV <= GRAD_NV)  // (its split makes no larger chunks)
            hipLaunchKernelGGL((k_distill_grad<T, NV>), dim3(grid), dim3(NT), 0, st, rows, k, sp, ids, stats, grad_loss,
                               static_cast<float>(tau), sc, grad);
    }
};

struct RowCall {
    Rows rows, grad;
    Teach te;
    int nvec;
    double tau;
    Scale sc;
    float *loss, *stats;
    const float *grad_loss;
    unsigned n;
    hipStream_t st;
    template <typename T, int NTB, int NV>
    void run() const
    {
        if (grad_loss)
            hipLaunchKernelGGL((k_distill_row<T, NTB, NV, true>), dim3(n), dim3(NTB), 0, st, rows, te, tau, sc,
                               loss, stats, grad_loss, grad);
        else
            hipLaunchKernelGGL((k_distill_row<T, NTB, NV, false>), dim3(n), dim3(NTB), 0, st, rows, te, tau, sc,
                               loss, stats, grad_loss, grad);
    }
    template <typename T>
    void pick() const
    {
        if (nvec <= 256 * 2)
            run<T, 256, 2>();
        else if (nvec <= 256 * 8)
            run<T, 256, 8>();
        else if (nvec <= 512 * 8)
            run<T, 512, 8>();
        else
            run<T, 1024, 8>();
    }
};

template <typename T, typename C>
void pick(const C &call)
{
    if (call.sp.nv <= 2)
        call.template run<T, 2>();
    else if (call.sp.nv <= 4)
        call.template run<T, 4>();
    else
        call.template run<T, 8>();
}

}  // namespace

namespace {

size_t parts_bytes(const domino_logits &lg)
{
    const size_t n = static_cast<size_t>(lg.B) * lg.R * split_of(lg, PART_NV).nch * sizeof(Part);
    return (n + 15) & ~static_cast<size_t>(15);
}

}  // namespace

size_t workspace_bytes(const domino_logits &lg, int k)
{
    if (whole_rows(lg, false))
        return 0;
    return parts_bytes(lg) + static_cast<size_t>(lg.B) * lg.R * (HEAD + k) * sizeof(float);
}

namespace {

// Loss, and gradient or statistics, in one launch.  False: not for these rows.
bool by_rows(const domino_logits &lg, const Teacher &t, double tau, const int32_t *n_rows, float *loss, float *stats,
             const float *grad_loss, const domino_logits *grad, hipStream_t st)
{
    RowCall c;
    if (!whole_rows(lg, grad_loss))
        return false;
    c.nvec = vectors(lg);
    c.rows = rows_of(lg, n_rows, n_rows != nullptr);
    c.grad = grad ? rows_of(*grad, nullptr, false) : Rows{};
    c.te = Teach{t.k, t.ids, t.values, t.lse};
    c.tau = tau;
    c.sc = scale_of(tau);
    c.loss = loss;
    c.stats = stats;
    c.grad_loss = grad_loss;
    c.n = static_cast<unsigned>(lg.B) * static_cast<unsigned>(lg.R);
    c.st = st;
    if (lg.dtype == DOMINO_F32)
        c.pick<float>();
    else
        c.pick<bf16s>();
    return true;
}

}  // namespace

namespace {

// keep: the logits may stay in the caches, for a gradient that follows.
hipError_t in_parts(const domino_logits &lg, const Teacher &t, double tau, const int32_t *n_rows, void *ws, float *loss,
                    float *stats, bool keep, hipStream_t st)
{
    PartCall c;
    c.rows = rows_of(lg, n_rows, n_rows != nullptr);
    c.te = Teach{t.k, t.ids, t.values, t.lse};
    c.sp = split_of(lg, PART_NV);
    c.sc = scale_of(tau);
    c.parts = static_cast<Part *>(ws);
    c.keep = keep;
    const unsigned n = static_cast<unsigned>(lg.B) * static_cast<unsigned>(lg.R);
    c.grid = n * c.sp.nch;
    c.st = st;
    if (lg.dtype == DOMINO_F32)
        pick<float>(c);
    else
        pick<bf16s>(c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (lg.dtype == DOMINO_F32)
        hipLaunchKernelGGL((k_distill_final<float>), dim3((n + NWAVE - 1) / NWAVE), dim3(NT), 0, st, c.rows, c.te,
                           static_cast<int>(n), c.sp.nch, tau, c.parts, loss, stats);
    else
        hipLaunchKernelGGL((k_distill_final<bf16s>), dim3((n + NWAVE - 1) / NWAVE), dim3(NT), 0, st, c.rows, c.te,
                           static_cast<int>(n), c.sp.nch, tau, c.parts, loss, stats);
    return hipGetLastError();
}

// Reading the logits so that the caches keep them, against passing the caches by, for rows of 151936, float32 (bfloat16
// alike): loss and gradient 80 against 87 us (156 MB), 115 against 123 (233 MB), 152 against 160 (311 MB), 229 against
// 234 (467 MB), 304.6 against 303.4 (622 MB); the loss alone 35 against 33, 48 against 44, 61 against 56, 87 against 79,
// 113 against 102.  So with the gradient up to twice the last-level cache's 256 MB, and without statistics never; with
// statistics the gradient is likely to follow but may not: up to 256 MB it gains as much as a loss without it would pay.
constexpr double KEEP_FOR_GRAD = 512e6, KEEP_FOR_STATS = 256e6;

double bytes_of(const domino_logits &lg)
{
    return static_cast<double>(lg.B) * lg.R * lg.V * (lg.dtype == DOMINO_F32 ? 4 : 2);
}

}  // namespace

hipError_t forward(const domino_logits &lg, const Teacher &t, double tau, const int32_t *n_rows, void *ws, float *loss,
                   float *stats, hipStream_t st)
{
    if (by_rows(lg, t, tau, n_rows, loss, stats, nullptr, nullptr, st))
        return hipGetLastError();
    return in_parts(lg, t, tau, n_rows, ws, loss, stats, stats && bytes_of(lg) <= KEEP_FOR_STATS, st);
}

hipError_t backward(const domino_logits &lg, int k, const int32_t *ids, const float *stats, const float *grad_loss,
                    double tau, const int32_t *n_rows, const domino_logits &grad, hipStream_t st)
{
    GradCall c;
    c.rows = rows_of(lg, n_rows, n_rows != nullptr);
    c.grad = rows_of(grad, nullptr, false);
    c.k = k;
    c.ids = ids;
    c.stats = stats;
    c.grad_loss = grad_loss;
    c.tau = tau;
    c.sp = split_of(lg, GRAD_NV);
    c.sc = scale_of(tau);
    c.grid = static_cast<unsigned>(lg.B) * static_cast<unsigned>(lg.R) * c.sp.nch;
    c.st = st;
    if (lg.dtype == DOMINO_F32)
        pick<float>(c);
    else
        pick<bf16s>(c);
    return hipGetLastError();
}

hipError_t both(const domino_logits &lg, const Teacher &t, double tau, const int32_t *n_rows, void *ws, float *loss,
                const float *grad_loss, const domino_logits &grad, hipStream_t st)
{
    if (by_rows(lg, t, tau, n_rows, loss, nullptr, grad_loss, &grad, st))
        return hipGetLastError();
    float *stats = reinterpret_cast<float *>(static_cast<char *>(ws) + parts_bytes(lg));
    const hipError_t e = in_parts(lg, t, tau, n_rows, ws, loss, stats, bytes_of(lg) <= KEEP_FOR_GRAD, st);
    return e == hipSuccess ? backward(lg, t.k, t.ids, stats, grad_loss, tau, n_rows, grad, st) : e;
}

}  // namespace dhdistill
