// Distillation from a teacher's kept top logits: the loss of a draft row
// against the teacher's K kept (id, logit) pairs, and its gradient.
//
// With q = softmax(z / T) over the draft row and teacher probabilities p_i on
// the kept ids,
//   loss = sum_i p_i (log p_i - log q_i) + p_r (log p_r - log q_r),
//   d loss / d z_v = (P q_v - p_v) / T              for a kept id v,
//                    (P q_v - p_r q_v / q_r) / T    for any other,
// where p_r is the teacher's mass outside the kept ids (from its log sum exp;
// 0 when the kept logits are renormalised), q_r the draft's, P = sum p_i + p_r.
// q_r is summed over the tokens outside the list alone, against their own
// maximum: 1 - sum q_i would lose it where the draft is sure.  A bitmap in
// shared memory marks the kept ids, which read as -inf in the sums.
//
// The loss streams a row once.  The gradient needs the row's sums before its
// first element; its kernel keeps the rows in flight in the shared memory of a
// cluster, so that it too reads them once.  The statistics are recomputed by the
// backward, nothing is kept between the calls.

#include <algorithm>
#include <atomic>

#include "grad_signals.cuh"
#include "kernels.h"
#include "row_slice.cuh"

namespace dspark {
namespace {

using namespace rows;

constexpr int kStreamThreads = 256;
constexpr float kNoRest = 1.0f / 1048576.0f;  // a teacher remainder below this counts as none

enum : int { kFlagBadToken = 1, kFlagNonfinite = 2, kFlagTimeout = 4, kFlagUsed = 8 };

struct alignas(16) Part {  // one CTA's sums: other tokens and kept ones, each against its own maximum
    float m_rest, rest, m_kept, kept;
    int flags;
};

struct Sums {  // a row's sums
    float m_rest, R, m, kept, S;  // R against m_rest, kept and S against m
    float t_max, t_sum, p_rest;
    int flags, code;
    bool taught, bad;
};

struct Row {  // a row's scalars, formed by one warp and read by all
    float m_rest;        // the other tokens' maximum
    float m;             // the row's
    float scale_rest;    // gradient of another token / its Scale(m_rest, a).exp_of(z)
    float scale_kept;    // P q / exp2((z - m) a)
    float t_max, inv_sum;  // the kept logits' maximum and 1 / sum (renormalised)
    float logs;          // log sum of the teacher less the draft's, in the units of loss
    float log_s, log_t;  // log of the sums alone, for the lowest values of the type
    float loss_rest;     // the remainder's term of the loss
    Sums sums;
};

struct EntrySums {  // the kept ids': logits of this slice, and the teacher's mass
    float m_kept, kept, t_max, t_sum;
    int flags;
};

template <int kWarps>
struct StreamShared {
    float top[kWarps], sum[kWarps];  // per warp: other tokens
    EntrySums entries[DSPARK_MAX_TOP / 32];  // per warp
    Part part;
    Row row;
    float loss_part[kMaxCluster][DSPARK_MAX_TOP / 32];  // rank 0's: every warp's share of the row's loss
    int last;
    double total[2][kWarps];
};

// y - log x for a positive finite x, good to 2^-23 of the result and of log 2:
// the exponent's share is taken off y first, in two parts of log 2 of which the
// first times an exponent is exact, so that nothing rounds at the size of log x.
__device__ __forceinline__ float minus_log(float y, float x) {
    constexpr float kHi = 0.693145751953125f, kLo = static_cast<float>(0.69314718055994531 - 0.693145751953125);
    int e;
    float f = frexpf(x, &e);  // [0.5, 1)
    if (f < 0.70710678f) {
        f *= 2.0f;
        e -= 1;
    }
    return (fmaf(-static_cast<float>(e), kHi, y) - static_cast<float>(e) * kLo) - log1pf(f - 1.0f);
}

// Rank 0 after its row's loss is written: counts the row and, if it was the
// last, sums the weighted losses and the weights of all rows in a fixed order.
template <int kThreads>
__device__ void finish_row(const DistillParams& p, StreamShared<kThreads / 32>& sh) {
    if (!p.loss_num) return;
    if (threadIdx.x == 0) sh.last = atom_add_acq_rel(p.ticket, 1u) == static_cast<unsigned>(p.N - 1);
    __syncthreads();
    if (!sh.last) return;
    double num = 0.0, den = 0.0;
    for (int64_t r = threadIdx.x; r < p.N; r += kThreads) {
        const float w = p.weight ? __ldg(p.weight + r) : 1.0f;
        if (w != 0.0f) num += static_cast<double>(w) * __ldcg(p.loss + r);
        den += w;
    }
    num = warp_sum(num);
    den = warp_sum(den);
    if ((threadIdx.x & 31) == 0) {
        sh.total[0][threadIdx.x >> 5] = num;
        sh.total[1][threadIdx.x >> 5] = den;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        num = join_sum(sh.total[0]);
        den = join_sum(sh.total[1]);
        if (threadIdx.x == 0) {
            p.loss_num[0] = static_cast<float>(num);
            p.loss_num[1] = static_cast<float>(den);
            *p.ticket = 0u;
        }
    }
}

template <int kDtype>
__device__ __forceinline__ void store_elem(char* p, float x) {
    if constexpr (kDtype == kBF16)
        *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
    else
        *reinterpret_cast<float*>(p) = x;
}

template <int kDtype>
__device__ __forceinline__ void store_vector(char* p, const float (&x)[Elem<kDtype>::kPer], bool aligned) {
    if (aligned) {
        uint4 v;
        if constexpr (kDtype == kBF16) {
            __nv_bfloat162 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            v = *reinterpret_cast<const uint4*>(b);
        } else {
            v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        }
        *reinterpret_cast<uint4*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < Elem<kDtype>::kPer; ++i) store_elem<kDtype>(p + i * Elem<kDtype>::kSize, x[i]);
    }
}

// Entry k of a row's list.
struct Entry {
    int id;
    float t;
};
// As it is loaded: bf16 logits are widened at their use, so that the load's
// result is not waited for before.
struct RawEntry {
    int id;
    uint32_t bits;
    __device__ __forceinline__ Entry widen(const DistillParams& p) const {
        return Entry{id, __uint_as_float(p.t_dtype == kBF16 ? bits << 16 : bits)};
    }
};
__device__ __forceinline__ RawEntry load_entry(const DistillParams& p, int64_t row, int k) {
    RawEntry e{-1, p.t_dtype == kBF16 ? 0xFF80u : 0xFF800000u};
    if (k < p.K) {
        const int64_t at = row * p.K + k;
        e.id = static_cast<int>(load_u32(p.index + at));
        e.bits = p.t_dtype == kBF16 ? load_u16(static_cast<const uint16_t*>(p.values) + at)
                                    : load_u32(static_cast<const uint32_t*>(p.values) + at);
    }
    return e;
}
// One warp: a row's entries into L2, ahead of their use (a line to a lane).
__device__ __forceinline__ void prefetch_entries(const DistillParams& p, int64_t row) {
    const int lane = threadIdx.x & 31, size = p.t_dtype == kBF16 ? 2 : 4;
    if (lane * 32 < p.K) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.index + row * p.K + lane * 32));
    if (lane * 128 < p.K * size)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p.values) + row * p.K * size + lane * 128));
}
__device__ __forceinline__ float load_weight(const DistillParams& p, int64_t row) {
    return p.weight ? load_f32(p.weight + row) : 1.0f;
}
__device__ __forceinline__ float load_lse(const DistillParams& p, int64_t row) { return p.lse ? load_f32(p.lse + row) : 0.0f; }
__device__ __forceinline__ int entry_flags(const DistillParams& p, const Entry& e) {
    if (e.id >= 0 && e.id < p.V) return kFlagUsed | (bad_logit(e.t) ? kFlagNonfinite : 0);
    return e.id != -1 ? kFlagBadToken : 0;
}
// log p_i, up to the renormalisation's sum.  t - T lse and t - t_max are formed
// before they are scaled: exact to 2^-23 of log p_i, not of t / T.
__device__ __forceinline__ float teacher_log(const DistillParams& p, float t, float lse, float t_max) {
    return p.lse ? fmaf(-p.t, lse, t) * p.inv_t : (t - t_max) * p.inv_t;
}

// One lane's entry added to its sums: its logit where the id is this slice's,
// and the teacher's where it is valid (-inf: without mass).
__device__ __forceinline__ void add_kept(EntrySums& q, float z, float a) {
    const float m = fmaxf(q.m_kept, z);  // passes a NaN over: the sum is NaN then
    q.kept = q.kept * ex2((q.m_kept - m) * a) + ex2((z - m) * a);
    q.m_kept = m;
}
__device__ __forceinline__ void add_teacher(const DistillParams& p, EntrySums& q, float t, float lse, float a) {
    if (!(t > neg_inf())) return;
    if (p.lse) {
        q.t_sum += expf(teacher_log(p, t, lse, 0.0f));
    } else {
        const float m = fmaxf(q.t_max, t);
        q.t_sum = q.t_sum * ex2((q.t_max - m) * a) + ex2((t - m) * a);
        q.t_max = m;
    }
}
// A warp's sums from its lanes'.
__device__ __forceinline__ void join_teacher(const DistillParams& p, EntrySums& q, float a) {
    if (p.lse)
        q.t_sum = warp_sum(q.t_sum);
    else
        join_lanes(q.t_max, q.t_sum, a);
}
__device__ __forceinline__ void join_kept(EntrySums& q, float a) {
    join_lanes(q.m_kept, q.kept, a);
    q.flags = __reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(q.flags));
}
constexpr EntrySums kNoEntries{kLowest, 0.0f, kLowest, 0.0f, 0};

// One warp, lane r with CTA r's part: the row's sums, and what the gradient
// needs of them (lane 0's are valid).
__device__ __forceinline__ void form_sums(const DistillParams& p, Part q, const EntrySums& e, float w, float lse, float a,
                                          Sums& g, Row& row) {
    g.flags = __reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(q.flags));
    join_lanes<kMaxCluster>(q.m_rest, q.rest, a);
    join_lanes<kMaxCluster>(q.m_kept, q.kept, a);
    g.t_max = e.t_max;
    g.t_sum = e.t_sum;
    g.m_rest = q.m_rest;
    g.R = q.rest;
    g.m = fmaxf(q.m_rest, q.m_kept);
    g.kept = q.kept * ex2((q.m_kept - g.m) * a);
    const float share = ex2((g.m_rest - g.m) * a);
    g.S = g.kept + g.R * share;
    g.taught = (g.flags & kFlagUsed) && (p.lse || g.t_sum > 0.0f);
    float mass = 1.0f;  // of the teacher: 1 but for rounding
    g.p_rest = 0.0f;
    if (p.lse) {
        g.p_rest = 1.0f - g.t_sum;
        if (!(g.p_rest >= kNoRest)) g.p_rest = 0.0f;
        mass = g.t_sum + g.p_rest;
        if (g.taught && !(fabsf(lse) < -neg_inf())) g.flags |= kFlagNonfinite;
    }
    g.code = g.flags & kFlagTimeout                     ? kReqTimeout
             : g.flags & kFlagBadToken                  ? kReqBadToken
             : (g.flags & kFlagNonfinite) || g.S != g.S ? kReqNonfinite
             : g.S == 0.0f || !g.taught                 ? kReqEmpty
                                                        : kReqOk;
    g.bad = g.code != kReqOk && (g.code != kReqEmpty || g.S == 0.0f);
    if ((threadIdx.x & 31) != 0) return;
    row.sums = g;
    row.m_rest = g.m_rest;
    row.m = g.m;
    row.t_max = g.t_max;
    row.inv_sum = p.lse ? 1.0f : g.taught ? 1.0f / g.t_sum : 0.0f;
    row.scale_kept = mass / g.S;
    const float c = mass * share / g.S - (g.p_rest > 0.0f && g.R > 0.0f ? g.p_rest / g.R : 0.0f);
    row.scale_rest = g.bad ? quiet_nan() : g.taught ? p.scale * w * p.inv_t * c * Scale(g.m_rest, a).remainder(g.m_rest) : 0.0f;
}

// One thread, row.sums standing: what the loss needs.  A loss is a small
// difference of logs: each is formed so that it rounds at the size of the
// difference.
__device__ __forceinline__ void form_loss(const DistillParams& p, float lse, Row& row) {
    const Sums& g = row.sums;
    const float s = g.bad ? 1.0f : g.S, t = g.t_sum > 0.0f ? g.t_sum : 1.0f;
    row.log_s = -minus_log(0.0f, s);
    row.log_t = p.lse ? 0.0f : -minus_log(0.0f, t);
    // T lse - m, like t_max - m, before it is scaled
    const float above = (p.lse ? fmaf(p.t, lse, -g.m) : g.t_max - g.m) * p.inv_t;
    row.logs = p.lse ? minus_log(above, s) : minus_log(above + row.log_t, s);
    float loss = 0.0f;
    if (g.p_rest > 0.0f && g.taught && !g.bad) {
        // log p_r - log q_r, both near 0 where nothing much is kept: each from
        // its complement there
        const float kept = g.kept / g.S, q_rest = g.R * ex2((g.m_rest - g.m) * (kLog2e * p.inv_t)) / g.S;
        const float log_q = kept < 0.5f        ? log1pf(-kept)
                            : q_rest > 1e-30f ? logf(q_rest)
                            : g.R > 0.0f      ? fmaf(g.m_rest - g.m, p.inv_t, logf(g.R) - row.log_s)
                                              : neg_inf();
        loss = g.p_rest * ((g.t_sum < 0.5f ? log1pf(-g.t_sum) : logf(g.p_rest)) - log_q);
    }
    row.loss_rest = loss;
}

// An entry's p_i, and its term of the loss where the id is this slice's:
// log p_i - log q_i is (t_i - z_i) / T less the difference of the two log sums
// (at the lowest values of the type, which t - z would lose them in, the logs
// themselves).
__device__ __forceinline__ float entry_term(const DistillParams& p, const Row& r, bool own, float z, float t, float lse,
                                            float& prob) {
    const float log_p = teacher_log(p, t, lse, r.t_max);
    prob = t > neg_inf() ? expf(log_p) * r.inv_sum : 0.0f;
    if (!own || !(prob > 0.0f)) return 0.0f;
    return prob * (fabsf(r.m) < 1e30f ? fmaf(t - z, p.inv_t, -r.logs)
                                      : (log_p - r.log_t) - fmaf(z - r.m, p.inv_t, -r.log_s));
}
__device__ __forceinline__ float entry_grad(const DistillParams& p, const Row& r, float w, float z, float prob, float a) {
    const float y = p.scale * w * p.inv_t * (r.scale_kept * ex2((z - r.m) * a) - prob);
    return r.sums.bad ? quiet_nan() : r.sums.taught ? y : 0.0f;
}

template <int kDtype>
__device__ __forceinline__ void zero_row(char* grow, const Slice<kDtype>& s, bool aligned, int threads) {
    constexpr int P = Elem<kDtype>::kPer, E = Elem<kDtype>::kSize;
    const float zero[P] = {};
    for (int j = threadIdx.x; j < s.count; j += threads)
        store_vector<kDtype>(grow + (static_cast<int64_t>(s.elem0) + j * P) * E, zero, aligned);
    const int e = s.edge_id();
    if (e >= 0) store_elem<kDtype>(grow + static_cast<int64_t>(e) * E, 0.0f);
}

// Rows streamed from memory: once for the loss, once more for the gradient of
// a row that no cluster can hold.  One cluster to a row.  Bound by the read: the
// loss of 7,168 bf16 rows of 129,280 takes 285 us, 1.86 GB at 6.5 TB/s, 0.96 of
// the measured copy bandwidth, with eight CTAs of 256 threads an SM (three of 512:
// 316 us; six of 256 with more registers: 298).
template <int kDtype, bool kGrad>
__global__ void __launch_bounds__(kStreamThreads, kGrad ? 4 : 8) distill_stream_kernel(const DistillParams p) {
    constexpr int P = Elem<kDtype>::kPer, E = Elem<kDtype>::kSize, kThreads = kStreamThreads, kWarps = kThreads / 32;
    static_assert(kThreads >= DSPARK_MAX_TOP, "an entry to a thread");
    extern __shared__ __align__(16) uint32_t s_drop[];
    __shared__ StreamShared<kWarps> sh;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x >> (__ffs(C) - 1);
    const Entry entry = load_entry(p, row, tid).widen(p);
    const float w = load_weight(p, row), lse = load_lse(p, row);
    const Slice<kDtype> s(p.draft, row, p.row_stride, p.V, rank, C);
    char* const grow = kGrad ? static_cast<char*>(p.grad) + row * p.V * E : nullptr;
    const bool aligned = kGrad && (reinterpret_cast<uintptr_t>(grow + static_cast<int64_t>(s.elem0) * E) & 15u) == 0;

    if (w == 0.0f) {  // a masked row: its logits are not read (the same branch in the whole cluster)
        if constexpr (kGrad) zero_row<kDtype>(grow, s, aligned, kThreads);
        if (rank == 0) {
            if (tid == 0) {
                p.loss[row] = 0.0f;
                p.status[row] = kReqOk;
            }
            finish_row<kThreads>(p, sh);
        }
        return;
    }

    StreamedRow<kDtype, kThreads> x(s);

    // ---- the bitmap of the kept ids, and their logits
    for (int i = tid; i < s.bitmap_words(); i += kThreads) s_drop[i] = 0u;
    int flags = entry_flags(p, entry);
    const bool valid = entry.id >= 0 && entry.id < p.V;
    const int b = valid ? s.bit_of(entry.id) : -1;
    const bool own = b >= 0;
    const float z = own ? load_elem<kDtype>(s.row + static_cast<int64_t>(entry.id) * E) : neg_inf();
    const float t = valid ? entry.t : neg_inf();
    __syncthreads();
    if (own && (atomicOr(&s_drop[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u)) flags |= kFlagBadToken;  // listed twice
    __syncthreads();
    x.set_drop(s_drop);

    // ---- maxima and sums of exp((x - max) / T), in powers of 2; -inf contributes 0
    const float a = kLog2e * p.inv_t;
    {
        const Running run = x.running(a);
        float m = run.m, sum = run.total(a);
        join_lanes(m, sum, a);
        if (lane == 0) {
            sh.top[warp] = m;
            sh.sum[warp] = sum;
        }
    }
    if (warp * 32 < p.K) {  // the same in the whole warp
        EntrySums q = kNoEntries;
        q.flags = flags;
        if (own) add_kept(q, z, a);
        add_teacher(p, q, t, lse, a);
        join_kept(q, a);
        join_teacher(p, q, a);
        if (lane == 0) sh.entries[warp] = q;
    }
    __syncthreads();
    EntrySums q = kNoEntries;
    if (warp == 0) {
        Part part;
        join_warps(sh.top, sh.sum, a, part.m_rest, part.rest);
        if (lane * 32 < p.K) q = sh.entries[lane];
        join_kept(q, a);
        join_teacher(p, q, a);
        part.m_kept = q.m_kept;
        part.kept = q.kept;
        part.flags = q.flags;
        if (lane == 0) sh.part = part;
        __syncwarp();
    }
    if (C > 1) cluster.sync();
    if (warp == 0) {
        Part part{kLowest, 0.0f, kLowest, 0.0f, 0};
        if (lane < C) part = C == 1 ? sh.part : *cluster.map_shared_rank(&sh.part, lane);
        Sums g;
        form_sums(p, part, q, w, lse, a, g, sh.row);
        if (lane == 0) form_loss(p, lse, sh.row);
    }
    __syncthreads();
    const Row& r = sh.row;

    // ---- the gradient: exp once more, then the kept ids over it
    if constexpr (kGrad) {
        const Scale scale(r.m_rest, a);
        x.each_batch([&](const auto& v, int j0) {
            constexpr int n = StreamedRow<kDtype, kThreads>::kBatch;
            float y[n][P];
            each_exp<kDtype>(v, scale, [&](int u, int i, uint64_t e) {
                split(mul2(e, pair(r.scale_rest, r.scale_rest)), y[u][2 * i], y[u][2 * i + 1]);
            });
#pragma unroll
            for (int u = 0; u < n; ++u)
                if (j0 + u * kThreads < s.count)
                    store_vector<kDtype>(grow + (static_cast<int64_t>(s.elem0) + (j0 + u * kThreads) * P) * E, y[u],
                                         aligned);
        });
        if (x.edge_at >= 0)
            store_elem<kDtype>(grow + static_cast<int64_t>(x.edge_at) * E, r.scale_rest * scale.exp_of(x.edge));
        __syncthreads();
    }
    if (warp * 32 < p.K) {
        float prob;
        const float term = warp_sum(entry_term(p, r, own, z, t, lse, prob));
        if (lane == 0) (C == 1 ? sh.loss_part : cluster.map_shared_rank(sh.loss_part, 0))[rank][warp] = term;
        if (kGrad && own)
            store_elem<kDtype>(grow + static_cast<int64_t>(entry.id) * E, entry_grad(p, r, w, z, prob, a));
    }
    sync(cluster, C);  // the shares have arrived; no CTA has left while another read its sums
    if (rank != 0) return;
    if (tid == 0) {
        float loss = r.loss_rest;
        for (int i = 0; i < C; ++i)
            for (int j = 0; j * 32 < p.K; ++j) loss += sh.loss_part[i][j];
        p.loss[row] = r.sums.bad ? quiet_nan() : r.sums.taught ? loss : 0.0f;
        p.status[row] = r.sums.code;
    }
    finish_row<kThreads>(p, sh);
}

// The gradient of rows whose slices fit shared memory three at a time.  Every
// cluster takes every clusters-th row; each CTA has two groups of workers and
// seven more warps.  The groups take the rows by turns, so that while one is in
// its first pass (maximum and sum of exp of each warp) or waits for the cluster
// to exchange a row's sums, the other is in its second (the gradient): loads,
// arithmetic and stores of two rows overlap, and a third row's slice is on its
// way into shared memory (one bulk copy).
//
// Warp D copies slices.  Two warps A let a row's kept ids read -inf in shared
// memory before the workers take it (their logits put aside).  Two warps B sum
// those, join the workers' sums, push the CTA's to every CTA of the cluster and
// form the row's scalars from all of them.  Two warps C, once a row's gradient is
// stored, store the kept ids' over it and push their share of the loss to rank 0,
// whose own write the row's loss two rows later.  Each pair takes the rows by
// turns too: a single warp's chain of latencies (2 to 3 us a row) would set the pace.
//
//   ready(n)    A -> workers       the slice is there, kept ids at -inf
//   entries(n)  A -> B             the kept ids' logits
//   sums(n)     workers -> B       the workers' sums
//   scalars(n)  B -> workers, C    the row's scalars
//   passed(n)   C -> A             the row is past them
//   stored(n)   workers -> C, D    the gradient is stored, the slice free
//
// Each is a named barrier in two sets, one for the rows of either parity.  A waits
// for passed(n) before it signals row n + 2: none is signalled again before all
// have passed it.  What orders the rows of one slice: grad_signals.cuh.
//
// Waits for copies and for other CTAs end after 2 s.  A CTA that gave one up goes
// through its remaining rows with the barriers above alone: it waits for nothing
// else, copies nothing and sends the others nothing, so that their waits end too;
// their rows from there on report DSPARK_REQ_TIMEOUT.  Before it ends, warp D waits
// again for the copies it had started, and the stores that others may have sent it
// are given time to arrive.
//
// Bound by memory: 7,168 bf16 rows of 129,280 take 547 us, 3.71 GB read and written
// at 6.8 TB/s, the measured copy bandwidth; 1,792 fp32 rows 292 us, 0.94 of it (a
// cluster of eight leaves some SMs idle).  Rows that lie otherwise within 16 bytes
// than the gradient's are stored element by element (the bf16 ones 2,209 us).  Before: one group of workers that did
// the two passes in turn, 702 us (the stores came in bursts); slices held in
// registers, 957; the gradient written over the logits and copied out in bulk, 779
// (the slice is occupied longer).
constexpr int kLosses = 8;  // rows whose shares of the loss may be on their way
constexpr int kSets = 4;    // rows between warps A's, the newest, and warps C's
constexpr uint64_t kLingerNs = 1000000;  // for the last stores sent to a CTA that gave up

struct Kept {  // an entry of the list on its way from warp A to warp C
    int id;    // of this slice, or -1
    float z, t;
};

struct Place {  // where a row's slice lies: vectors in it, its first element, the row's edge
    int count, elem0, head, tail0;
};

template <int kGroupWarps>
struct GradShared {
    uint64_t full[kFull];       // a row's slice has arrived
    uint64_t parts_in[4];       // every CTA's part has
    uint64_t loss_in[kLosses];  // rank 0's: every CTA's share of the loss has
    Part part[4][kMaxCluster];
    float loss_part[kLosses][kMaxCluster];
    float top[2][kGroupWarps], sum[2][kGroupWarps];
    int flags[4][32];  // warp A's lanes'
    Row row[4];
    float weight[4];
    float edge[kSlices][16];  // the row's edge: its head, from 8 on its tail
    Place place[4];
    int timeout;
};

enum : int { kBarReady = 1, kBarEntries = 3, kBarSums = 5, kBarScalars = 7, kBarStored = 9, kBarPassed = 11 };

// Whether a wait of this CTA was given up (the same answer in the whole warp).
__device__ __forceinline__ bool gave_up(const int& timeout) {
    return __any_sync(0xFFFFFFFFu, *const_cast<const volatile int*>(&timeout));
}

template <int kDtype, int kWorkers, int kNV>
constexpr int grad_smem(int K) {
    constexpr int slice = kNV * (kWorkers / 2) * 16;
    return kSlices * slice + 2 * (slice / Elem<kDtype>::kSize / 32 + 1) * 4 + (kSets + 2) * K * static_cast<int>(sizeof(Kept));
}

template <int kDtype, int kWorkers, int kNV, int kCtas>
__global__ void __launch_bounds__(kWorkers + 224, kCtas) distill_grad_kernel(const DistillParams p) {
    constexpr int P = Elem<kDtype>::kPer, E = Elem<kDtype>::kSize;
    constexpr int kGradThreads = kWorkers + 224, kGradWarps = kWorkers / 32;
    constexpr int kGroup = kWorkers / 2, kGroupWarps = kGradWarps / 2;  // workers of the rows of one parity
    constexpr int kSliceBytes = kNV * (kWorkers / 2) * 16;
    // kSlices slices, for each warp A a bit per element (to find an id listed
    // twice), the lists on their way from warps A to warps C, and those at warps A
    extern __shared__ __align__(128) char s_dyn[];
    constexpr int kMarkWords = kSliceBytes / E / 32 + 1;
    __shared__ __align__(16) GradShared<kGroupWarps> sh;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = blockIdx.x >> (__ffs(C) - 1), step = gridDim.x >> (__ffs(C) - 1);
    const int rows = static_cast<int>((p.N - row0 + step - 1) / step);  // of this cluster: at least one
    const float a = kLog2e * p.inv_t;

    if (tid == 0) {
        for (int i = 0; i < kFull; ++i) mbar_init(&sh.full[i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&sh.parts_in[i], 1);
        for (int i = 0; i < kLosses; ++i) mbar_init(&sh.loss_in[i], 1);
        fence_mbar_init();
        sh.timeout = 0;
    }
    uint32_t* const s_marks = reinterpret_cast<uint32_t*>(s_dyn + kSlices * kSliceBytes);
    Kept* const s_kept = reinterpret_cast<Kept*>(s_marks + 2 * kMarkWords);
    Kept* const s_list = s_kept + kSets * p.K;
    for (int i = tid; i < 2 * kMarkWords; i += kGradThreads) s_marks[i] = 0u;
    sync(cluster, C);

    if (warp < kGradWarps) {
        // ------------------------------------------------------------ workers
        const int own = warp / kGroupWarps, t = tid - own * kGroup;  // takes the rows of this parity
        const int edge_slot = (t & 7) + (t & 32) / 4;
#pragma unroll 1
        for (int n = own; n < rows; n += 2) {
            uint4* const slice = reinterpret_cast<uint4*>(s_dyn + slice_of(n) * kSliceBytes);
            bar_sync(kBarReady + own, kGroup + 32);
            const Place g = sh.place[n & 3];
            const bool masked = sh.weight[n & 3] == 0.0f;
            // this thread's element of the edge, if it holds one (threads 0..7 and 32..39 of rank 0)
            int edge_at = -1;
            if (rank == 0) edge_at = t < g.head ? t : t >= 32 && t - 32 < p.V - g.tail0 ? g.tail0 + t - 32 : -1;
            const float edge = edge_at >= 0 ? sh.edge[slice_of(n)][edge_slot] : neg_inf();
            if (!masked) {
                constexpr int kBatch = kNV < 8 ? kNV : 8;
                Running run;
#pragma unroll 1
                for (int j0 = t; (j0 & ~31) < g.count; j0 += kBatch * kGroup) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        v[u] = j0 + u * kGroup < g.count ? slice[j0 + u * kGroup] : neg_inf_vector<kDtype>();
                    run.add<kDtype>(v, vector_max<kDtype>(v), a);
                }
                if (edge_at >= 0) run.add(edge, a);
                float m = run.m, sum = run.total(a);
                join_lanes(m, sum, a);
                if (lane == 0) {
                    sh.top[own][warp % kGroupWarps] = m;
                    sh.sum[own][warp % kGroupWarps] = sum;
                }
            }
            bar_arrive(kBarSums + own, kGroup + 32);
            char* const grow = static_cast<char*>(p.grad) + (row0 + n * step) * p.V * E;
            char* const out = grow + static_cast<int64_t>(g.elem0) * E;
            const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
            bar_sync(kBarScalars + own, kGroup + 64);
            if (masked) {
                const float zero[P] = {};
                for (int j = t; j < g.count; j += kGroup)
                    store_vector<kDtype>(out + static_cast<int64_t>(j) * 16, zero, aligned);
                if (edge_at >= 0) store_elem<kDtype>(grow + static_cast<int64_t>(edge_at) * E, 0.0f);
            } else {
                const float c = sh.row[n & 3].scale_rest;
                const Scale scale(sh.row[n & 3].m_rest, a);
                constexpr int kBatch = kNV < 4 ? kNV : 4;
#pragma unroll 1
                for (int j0 = t; j0 < g.count; j0 += kBatch * kGroup) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        v[u] = j0 + u * kGroup < g.count ? slice[j0 + u * kGroup] : neg_inf_vector<kDtype>();
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        const uint4 one[1] = {v[u]};
                        float y[P];
                        each_exp<kDtype>(one, scale, [&](int, int i, uint64_t e) {
                            split(mul2(e, pair(c, c)), y[2 * i], y[2 * i + 1]);
                        });
                        if (j0 + u * kGroup < g.count)
                            store_vector<kDtype>(out + static_cast<int64_t>(j0 + u * kGroup) * 16, y, aligned);
                    }
                }
                if (edge_at >= 0) store_elem<kDtype>(grow + static_cast<int64_t>(edge_at) * E, c * scale.exp_of(edge));
            }
            bar_arrive(kBarStored + own, kGroup + 64);
        }
    } else if (warp < kGradWarps + 2) {
        // ------------------------------------------------------------ warps A
        // (loops of a few instructions: unrolled, they would crowd the workers' code
        // out of the instruction caches)
        const int own = warp - kGradWarps;  // takes the rows of this parity
        uint32_t* const s_mark = s_marks + own * kMarkWords;
#pragma unroll 1
        for (int n = own; n < rows; n += 2) {
            const int at = slice_of(n);
            const int64_t row = row0 + n * step;
            const Slice<kDtype> s(p.draft, row, p.row_stride, p.V, rank, C);
            const float w = load_weight(p, row);
            if (n + 2 < rows) prefetch_entries(p, row + 2 * step);
            // ---- what does not need the slice: where its kept ids are
            float edge_value = neg_inf();  // lanes 0..7 the edge's head, 8..15 its tail
            if (rank == 0 && lane < 16 && w != 0.0f) {
                const int id = lane < 8 ? lane : s.tail0 + lane - 8;
                if (id < (lane < 8 ? s.head : s.V)) edge_value = load_elem<kDtype>(s.row + static_cast<int64_t>(id) * E);
            }
            Kept* const list = s_list + own * p.K;  // this warp's, z still the bits of where the logit is
            int flags = 0;
#pragma unroll 2
            for (int k = lane; k < p.K; k += 32) {
                const Entry e = load_entry(p, row, k).widen(p);
                const bool valid = e.id >= 0 && e.id < p.V;
                const int b = valid ? s.bit_of(e.id) : -1;
                flags |= entry_flags(p, e);
                if (b >= 0 && (atomicOr(&s_mark[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u)) flags |= kFlagBadToken;  // twice
                list[k] = Kept{b >= 0 ? e.id : -1, __int_as_float(b), valid ? e.t : neg_inf()};
            }
            __syncwarp();
#pragma unroll 1
            for (int k = lane; k < p.K; k += 32) {
                const int b = __float_as_int(list[k].z);
                if (b >= 0) s_mark[b >> 5] = 0u;
            }
            // row n - 2 is past its scalars: all have passed what is signalled below
            if (n > 1) bar_sync(kBarPassed + own, 64);
            if (!gave_up(sh.timeout) && !mbar_wait(&sh.full[full_of(n)], full_parity(n), kWaitLimitNs)) sh.timeout = 1;
            __syncwarp();
            // ---- the slice is there
            float* const edge = sh.edge[at];
            if (lane < 16) edge[lane] = edge_value;
            if (lane == 0) {
                sh.weight[n & 3] = w;
                sh.place[n & 3] = Place{s.count, s.elem0, s.head, s.tail0};
            }
            sh.flags[n & 3][lane] = flags;
            __syncwarp();
            if (w != 0.0f) {
                char* const slice = s_dyn + at * kSliceBytes;
                Kept* const kept = s_kept + (n & (kSets - 1)) * p.K;
                const int edge0 = s.edge_word() * 32;
                // a kept id's logit put aside, -inf in its place (an id listed twice
                // may find that already: its row fails)
#pragma unroll 2
                for (int k = lane; k < p.K; k += 32) {
                    Kept e = list[k];
                    const int b = __float_as_int(e.z);
                    e.z = neg_inf();
                    if (b >= edge0) {
                        e.z = edge[b & 15];
                        edge[b & 15] = neg_inf();
                    } else if (b >= 0) {
                        if constexpr (kDtype == kBF16) {
                            uint16_t* const x = reinterpret_cast<uint16_t*>(slice) + b;
                            e.z = __uint_as_float(static_cast<uint32_t>(*x) << 16);
                            *x = 0xFF80u;
                        } else {
                            float* const x = reinterpret_cast<float*>(slice) + b;
                            e.z = *x;
                            *x = neg_inf();
                        }
                    }
                    kept[k] = e;
                }
                fence_proxy_async_smem();  // before the next copy writes here
            }
            __syncwarp();
            bar_arrive(kBarReady + own, kGroup + 32);
            bar_arrive(kBarEntries + own, 64);
        }
    } else if (warp < kGradWarps + 4) {
        // ------------------------------------------------------------ warps B
        const int own = warp - kGradWarps - 2;
        uint32_t phase = 0;  // bit i: the parity of sh.parts_in[i]
        float w_next = 0.0f, lse_next = 0.0f;
        auto load_row = [&](int n) {
            if (n >= rows) return;
            w_next = load_weight(p, row0 + n * step);
            lse_next = load_lse(p, row0 + n * step);
        };
        load_row(own);
#pragma unroll 1
        for (int n = own; n < rows; n += 2) {
            const int i = n & 3;
            const float w = w_next, lse = lse_next;
            load_row(n + 2);
            const bool expected = !gave_up(sh.timeout);
            if (expected && lane == 0) mbar_arrive_expect_tx(&sh.parts_in[i], C * 20);
            EntrySums q = kNoEntries;
            if (w != 0.0f) {  // the teacher's sums need no slice
#pragma unroll 2
                for (int k = lane; k < p.K; k += 32) {
                    const Entry e = load_entry(p, row0 + n * step, k).widen(p);
                    add_teacher(p, q, e.id >= 0 && e.id < p.V ? e.t : neg_inf(), lse, a);
                }
                join_teacher(p, q, a);
            }
            bar_sync(kBarEntries + own, 64);
            if (w != 0.0f) {
                q.flags = sh.flags[i][lane];
#pragma unroll 1
                for (int k = lane; k < p.K; k += 32) {
                    const Kept e = s_kept[(n & (kSets - 1)) * p.K + k];
                    if (e.id >= 0) add_kept(q, e.z, a);
                }
                join_kept(q, a);
            }
            bar_sync(kBarSums + own, kGroup + 32);
            // masked rows too: the exchange keeps the cluster's CTAs within two rows of each other
            Part part;
            part.m_rest = sh.top[own][lane & (kGroupWarps - 1)];
            part.rest = sh.sum[own][lane & (kGroupWarps - 1)];
            join_lanes<kGroupWarps>(part.m_rest, part.rest, a);
            part.flags = q.flags;
            if (!gave_up(sh.timeout) && lane < C) {
                const uint32_t dst = cluster_addr(&sh.part[i][rank], lane), bar = cluster_addr(&sh.parts_in[i], lane);
                push_v4(dst, part.m_rest, part.rest, q.m_kept, q.kept, bar);
                push_u32(dst + 16, static_cast<uint32_t>(part.flags), bar);
            }
            if (!gave_up(sh.timeout) && !mbar_wait_cluster(&sh.parts_in[i], phase >> i & 1u, kWaitLimitNs)) sh.timeout = 1;
            phase ^= 1u << i;
            __syncwarp();
            part = Part{kLowest, 0.0f, kLowest, 0.0f, 0};
            if (lane < C) part = sh.part[i][lane];
            if (gave_up(sh.timeout)) part.flags |= kFlagTimeout;
            Sums g;
            form_sums(p, part, q, w, lse, a, g, sh.row[i]);
            __syncwarp();
            bar_arrive(kBarScalars + own, kGroup + 64);
        }
    } else if (warp < kGradWarps + 6) {
        // ------------------------------------------------------------ warps C
        const int own = warp - kGradWarps - 4;
        uint32_t phase = 0;      // bit i: the parity of sh.loss_in[i]
        int64_t last_row = -1;   // this warp's last row, whose shares may still be on their way (-1: none)
        auto write_loss = [&](int n) {
            if (rank != 0 || last_row < 0) return;
            const int i = n & (kLosses - 1);
            if (!gave_up(sh.timeout) && !mbar_wait_cluster(&sh.loss_in[i], phase >> i & 1u, kWaitLimitNs)) sh.timeout = 1;
            phase ^= 1u << i;
            __syncwarp();
            const bool late = gave_up(sh.timeout);
            if (lane == 0) {
                const Row& r = sh.row[n & 3];
                float loss = r.loss_rest;
                for (int k = 0; k < C; ++k) loss += sh.loss_part[i][k];
                p.loss[last_row] = r.sums.bad || late ? quiet_nan() : r.sums.taught ? loss : 0.0f;
                p.status[last_row] = late ? kReqTimeout : r.sums.code;
            }
            __syncwarp();
        };
        float w_next = 0.0f, lse_next = 0.0f;
        auto load_row = [&](int n) {
            if (n >= rows) return;
            w_next = load_weight(p, row0 + n * step);
            lse_next = load_lse(p, row0 + n * step);
        };
        load_row(own);
        int n = own;
#pragma unroll 1
        for (; n < rows; n += 2) {
            const int64_t row = row0 + n * step;
            const float w = w_next, lse = lse_next;
            load_row(n + 2);
            const int turn = n & (kLosses - 1);
            const bool expecting = rank == 0 && w != 0.0f && !gave_up(sh.timeout);
            if (expecting && lane == 0) mbar_arrive_expect_tx(&sh.loss_in[turn], C * 4);
            write_loss(n - 2);
            bar_sync(kBarScalars + own, kGroup + 64);
            if (n + 2 < rows) bar_arrive(kBarPassed + own, 64);
            Row& r = sh.row[n & 3];
            if (lane == 0 && w != 0.0f) form_loss(p, lse, r);
            __syncwarp();
            bar_sync(kBarStored + own, kGroup + 64);
            if (w != 0.0f) {
                char* const grow = static_cast<char*>(p.grad) + row * p.V * E;
                float term = 0.0f;
#pragma unroll 1
                for (int k = lane; k < p.K; k += 32) {
                    const Kept e = s_kept[(n & (kSets - 1)) * p.K + k];
                    if (e.id < 0) continue;
                    float prob;
                    term += entry_term(p, r, true, e.z, e.t, lse, prob);
                    store_elem<kDtype>(grow + static_cast<int64_t>(e.id) * E, entry_grad(p, r, w, e.z, prob, a));
                }
                term = warp_sum(term);
                if (!gave_up(sh.timeout) && lane == 0)
                    push_u32(cluster_addr(&sh.loss_part[turn][rank], 0), __float_as_uint(term),
                             cluster_addr(&sh.loss_in[turn], 0));
            } else if (rank == 0 && lane == 0) {
                p.loss[row] = 0.0f;
                p.status[row] = kReqOk;
            }
            last_row = w != 0.0f ? row : -1;
        }
        write_loss(n - 2);
    } else {
        // ------------------------------------------------------------- warp D
        int begun = 0;  // rows announced
        // one arrival on the row's mbarrier, with or without a copy
        auto copy = [&](int n, float w) {
            if (n >= rows || gave_up(sh.timeout) || lane != 0) return;
            begun = n + 1;
            const Slice<kDtype> s(p.draft, row0 + n * step, p.row_stride, p.V, rank, C);
            uint64_t* const full = &sh.full[full_of(n)];
            if (w == 0.0f || s.count == 0) {
                mbar_arrive(full);
                return;
            }
            mbar_arrive_expect_tx(full, s.count * 16);
            bulk_g2s(s_dyn + slice_of(n) * kSliceBytes, s.vec(0), s.count * 16, full);
        };
        auto weight = [&](int n) { return n < rows ? load_weight(p, row0 + n * step) : 0.0f; };
        copy(0, weight(0));
        copy(1, weight(1));
        copy(2, weight(2));
        float w_next = weight(3);
#pragma unroll 1
        for (int n = 0; n < rows; ++n) {
            const float w = w_next;
            w_next = weight(n + 4);
            bar_sync(kBarStored + (n & 1), kGroup + 64);  // the slice of row n is free
            copy(n + 3, w);
        }
        // copies that nobody waited for may still be in flight: this shared memory is their target
        if (gave_up(sh.timeout))
            for (int n = max(0, begun - kFull); n < begun; ++n)
                mbar_wait(&sh.full[full_of(n)], full_parity(n), kWaitLimitNs);
    }
    __syncwarp();
    if (C > 1) cluster.sync();  // no CTA leaves while another may still push to it
    if (gave_up(sh.timeout)) {  // nor before what was pushed, and not waited for, is there
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kLingerNs) {}
    }
}

// Clusters of C CTAs of a kernel that can be resident at once (0 if the query fails).
template <class K>
int resident(K kernel, int C, int threads, size_t smem) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kernel), &cfg) == cudaSuccess ? n : 0;
}

template <int kDtype, int kWorkers, int kNV, int kCtas>
cudaError_t launch_held(const DistillParams& p, int C, cudaStream_t stream) {
    const auto kernel = distill_grad_kernel<kDtype, kWorkers, kNV, kCtas>;
    const int smem = grad_smem<kDtype, kWorkers, kNV>(p.K);
    // per device, cluster size and length of the lists in 64s: the clusters
    // resident at once (0: not yet queried; host threads may race here)
    static std::atomic<int> cache[64][4][DSPARK_MAX_TOP / 64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int ci = C == 1 ? 0 : C == 2 ? 1 : C == 4 ? 2 : 3, lists = (p.K - 1) / 64;
    int n = dev < 64 ? cache[dev][ci][lists].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 grad_smem<kDtype, kWorkers, kNV>(DSPARK_MAX_TOP));
        if (e != cudaSuccess) return e;
        n = resident(kernel, C, kWorkers + 224, grad_smem<kDtype, kWorkers, kNV>(64 * (lists + 1)));
        if (n <= 0) return cudaErrorInvalidConfiguration;
        if (dev < 64) cache[dev][ci][lists].store(n, std::memory_order_release);
    }
    return launch_row_kernel(kernel, std::min<int64_t>(p.N, n), C, kWorkers + 224, smem, stream, p);
}

template <int kDtype, bool kGrad>
cudaError_t launch_streamed(const DistillParams& p, cudaStream_t stream) {
    const int C = spread(p.N, p.V / Elem<kDtype>::kPer, kStreamThreads, 64, kStreamFill);
    const size_t smem = static_cast<size_t>(max_bitmap_words(p.V, C)) * sizeof(uint32_t);
    return launch_row_kernel(distill_stream_kernel<kDtype, kGrad>, p.N, C, kStreamThreads, smem, stream, p);
}

// Slices of up to 16 vectors a thread of a group.  Small ones leave room for two
// CTAs of 128-thread groups an SM, which hide each other's chains of latencies
// (4,096 rows of 16,000 bf16 logits 56 us, against 77 with one CTA of 256-thread
// groups; 8,192 rows of 4,096 fp32 ones 75 against 119; 8,192 rows of 4,096 bf16
// ones 70, against 82 in batches of eight).  Rows that would take more CTAs
// for it are not split (32,003 bf16 logits: 92 us on one CTA, 97 on two), and
// with longer lists the 16-vector slices do not fit twice.  Rows of more than
// 32,768 vectors are streamed twice: half of that long, held rows win by 1.5
// (131,072 vectors: 184 us against 270 for 1,000 rows).
template <int kDtype>
cudaError_t launch_grad(const DistillParams& p, cudaStream_t stream) {
    const int64_t vectors = p.V / Elem<kDtype>::kPer;
    int C = spread(p.N, vectors, 256, 8, kSms);
    if (vectors <= static_cast<int64_t>(C) * 4 * 128) return launch_held<kDtype, 256, 4, 2>(p, C, stream);
    if (vectors <= static_cast<int64_t>(C) * 8 * 128) return launch_held<kDtype, 256, 8, 2>(p, C, stream);
    if (vectors <= 16 * 128 && p.K <= 96) return launch_held<kDtype, 256, 16, 2>(p, C, stream);
    C = spread(p.N, vectors, 512, 8, kSms);
    if (vectors <= static_cast<int64_t>(C) * 16 * 256) return launch_held<kDtype, 512, 16, 1>(p, C, stream);
    return launch_streamed<kDtype, true>(p, stream);
}

}  // namespace

cudaError_t launch_distill(const DistillParams& p, cudaStream_t stream) {
    if (p.grad) return p.dtype == kBF16 ? launch_grad<kBF16>(p, stream) : launch_grad<kF32>(p, stream);
    return p.dtype == kBF16 ? launch_streamed<kBF16, false>(p, stream) : launch_streamed<kF32, false>(p, stream);
}

}  // namespace dspark
