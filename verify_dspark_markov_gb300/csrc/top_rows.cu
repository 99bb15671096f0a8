// The best entries of vocabulary rows: a teacher's kept top logits with the
// row's log sum exp, and beam search's selection over beams and vocabulary.
//
// Every entry has a 64-bit key, its value's order-preserving bits above the
// complement of its index, so that keys are distinct and the larger key is the
// larger value, or the lower index at equal values.  The k best are the keys
// above a floor found by histograms over ever narrower key ranges: the range
// is cut into 256 bins, the bin that holds the k-th key becomes the range,
// and the search stops once the keys above its lower end fit the candidate
// buffer.  The row is read once, keeping the maximum of each group of eight
// vectors (four of each of two neighbouring threads: whole 32-byte sectors)
// beside the running sum of exp; a first search over the groups' maxima
// gives a floor with at least k entries above it and seldom many more, and only
// the groups that reach it are read again.  If they overflow the buffer (rows
// of equal values) a search over all entries follows.  The candidates are then
// ranked by counting larger ones.
//
// Beam search ranks s_w + ((z - max) - log sum exp(z - max)), rounded in that
// order in 32 bits, which is monotone in z: the same search runs on the
// scores.  Each beam's m best go to the workspace; the last beam of an item to
// arrive merges them.
//
// What bounds it: the row's one read (the top 64 of 8,192 bf16 rows of 129,280:
// 357 us, 2.12 GB at 5.95 TB/s, 0.88 of the measured copy bandwidth).  The groups
// read again add 8 % (DRAM hands out 64 bytes for 32), and a row's search is a
// chain of barriers in which its CTA loads nothing; so CTAs are small, 256 threads
// and six of them an SM (512 threads and three: 406 us), and the others' loads
// cover it.  Few rows are bound by that chain: 4 us of the 8 to 10 that one
// request's rows or beams take on the device.

#include "kernels.h"
#include "row_slice.cuh"

namespace dspark {
namespace {

using namespace rows;

constexpr int kThreads = 256, kBinBits = 8;  // a bin to a thread
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 1024;  // candidates ranked at the end
constexpr int kBatch = 4;   // vectors a thread reads at a time
constexpr int kPairs = kThreads / 2;
constexpr int kBatches = 32;  // such batches of a slice at most
constexpr uint64_t kFirstKey = 0x00800000ull << 32;  // below every value but -inf
constexpr uint64_t kFailed = ~0ull;                  // a list's mark for a row that cannot be ranked

__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
    return static_cast<uint64_t>(ordered_key(v)) << 32 | (0xFFFFFFFFu - index);
}

struct TopShared {
    uint32_t hist[3][kThreads];  // used in turn: one filled, one cleared, one maybe still read
    uint32_t total[kThreads];    // the bins of all CTAs
    uint32_t pick_bin, pick_above, pick_count;
    float red[3][kWarps];
    float part[3];               // this CTA's maximum, sum of exp, least of the threads' maxima
    uint32_t count;              // rank 0's: candidates
    uint64_t cand[kCap];
    float group[kBatches * kPairs];  // the groups' maxima
    uint16_t reach[kCap];            // the groups that reach the floor
    uint32_t reached;
    int last;
};

// The lower end of a range [floor, hi) that holds at least `want` of the keys
// each() visits in [lo, hi), and no more than `cap` of them unless keys agree in
// all but their lowest `equal` bits; 0 if there are fewer than `want`.
template <class Each>
__device__ uint64_t find_floor(Each each, uint32_t want, uint32_t cap, int equal, uint64_t lo, uint64_t hi,
                               TopShared& sh, int& turn, const cg::cluster_group& cluster, int C) {
    const int tid = threadIdx.x;
    uint32_t above = 0;
    while (true) {
        const uint64_t span = hi - lo - 1;
        const int shift = span >> kBinBits ? 64 - kBinBits - __clzll(span) : 0;
        uint32_t* const h = sh.hist[turn % 3];
        sh.hist[(turn + 1) % 3][tid] = 0;
        ++turn;
        each([&](uint64_t key) {
            if (key >= lo && key < hi) atomicAdd(&h[(key - lo) >> shift], 1u);
        });
        sync(cluster, C);
        const uint32_t* bins = h;
        if (C > 1) {
            uint32_t n = 0;
            for (int r = 0; r < C; ++r) n += ld_cluster(cluster_addr(&h[tid], r));
            sh.total[tid] = n;
            bins = sh.total;
            __syncthreads();
        }
        if (tid < 32) {  // one warp finds the bin of the want-th key, eight bins to a lane from the top down
            constexpr int kPer = kThreads / 32;
            uint32_t n[kPer], sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                n[i] = bins[kThreads - 1 - tid * kPer - i];
                sum += n[i];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (tid >= o) incl += y;
            }
            uint32_t before = above + incl - sum;
            const bool here = before < want && before + sum >= want;
            if (here) {
                int i = 0;
#pragma unroll
                for (int q = 0; q < kPer - 1; ++q)
                    if (i == q && before + n[q] < want) {
                        before += n[q];
                        ++i;
                    }
                uint32_t count = 0;
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (i == q) count = n[q];
                sh.pick_bin = kThreads - 1 - tid * kPer - i;
                sh.pick_above = before;
                sh.pick_count = count;
            }
            if (!__any_sync(0xFFFFFFFFu, here) && tid == 0) sh.pick_count = 0;
        }
        __syncthreads();
        if (sh.pick_count == 0) return 0;
        lo += static_cast<uint64_t>(sh.pick_bin) << shift;
        hi = min(hi, lo + (uint64_t(1) << shift));
        above = sh.pick_above;
        if (above + sh.pick_count <= cap || shift <= equal) return lo;
    }
}

// The candidates in sh.cand ranked by counting: f(rank, key) for the first k.
template <class F>
__device__ __forceinline__ void rank_candidates(const TopShared& sh, int count, int k, F f) {
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const uint64_t key = sh.cand[i];
        int r = 0;
        for (int j = 0; j < count; ++j) r += sh.cand[j] > key;
        if (r < k) f(r, key);
    }
}

// The keys at or above `floor` that each() visits, into rank 0's buffer.
// Returns their number in every thread (it may exceed the buffer).
template <class Each>
__device__ int gather(Each each, uint64_t floor, TopShared& sh, const cg::cluster_group& cluster, int C) {
    const int leader = C == 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const uint32_t count = cluster_addr(&sh.count, leader), cand = cluster_addr(sh.cand, leader);
    each([&](uint64_t key) {
        if (key >= floor) {
            const uint32_t at = atom_add_cluster(count, 1u);
            if (at < kCap) st_cluster(cand + at * 8, key);
        }
    });
    sync(cluster, C);
    return static_cast<int>(ld_cluster(count));
}

// Beam search: the last beam of item b to arrive merges the lists.
__device__ void merge_beams(const TopParams& p, int64_t b, TopShared& sh, int& turn,
                            const cg::cluster_group& cluster) {
    const int tid = threadIdx.x;
    const int n = p.W * p.k;
    const uint64_t* const list = p.lists + b * n;
    bool failed = false;
    auto each = [&](auto f) {
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t key = __ldcg(reinterpret_cast<const unsigned long long*>(list + i));
            if (key == kFailed)
                failed = true;
            else if (key)
                f(key);
        }
    };
    if (tid == 0) sh.count = 0;
    __syncthreads();
    uint64_t floor = kFirstKey;
    if (n > kCap) floor = max(kFirstKey, find_floor(each, p.k, kCap, 0, kFirstKey, kFailed, sh, turn, cluster, 1));
    const int count = gather(each, floor, sh, cluster, 1);
    failed = __syncthreads_or(failed);
    auto put = [&](int r, float score, int parent, int token) {
        p.out_score[b * p.k + r] = score;
        p.out_parent[b * p.k + r] = parent;
        p.out_token[b * p.k + r] = token;
    };
    for (int r = (failed ? 0 : count) + tid; r < p.k; r += kThreads) put(r, failed ? quiet_nan() : neg_inf(), -1, -1);
    if (!failed)
        rank_candidates(sh, count, p.k, [&](int r, uint64_t key) {
            const uint32_t flat = 0xFFFFFFFFu - static_cast<uint32_t>(key);
            put(r, key_to_float(static_cast<uint32_t>(key >> 32)), flat / p.V, flat % p.V);
        });
    if (tid == 0) {
        p.status[b] = failed ? kReqNonfinite : count ? kReqOk : kReqEmpty;
        p.ticket[b] = 0u;
    }
}

// After a beam's list is written by rank 0.
__device__ void finish_beam(const TopParams& p, int64_t row, TopShared& sh, int& turn,
                            const cg::cluster_group& cluster) {
    const int64_t b = row / p.W;
    __syncthreads();
    if (threadIdx.x == 0) sh.last = atom_add_acq_rel(p.ticket + b, 1u) == static_cast<unsigned>(p.W - 1);
    __syncthreads();
    if (sh.last) merge_beams(p, b, sh, turn, cluster);
}

template <int kDtype, bool kBeam>
__global__ void __launch_bounds__(kThreads, 6) top_kernel(const TopParams p) {
    constexpr int P = Elem<kDtype>::kPer;
    __shared__ TopShared sh;

    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / C;
    int turn = 0;
    sh.hist[0][tid] = 0;
    if (tid == 0) sh.count = sh.reached = 0;

    float base = 0.0f;     // the beam's score so far
    uint32_t index0 = 0;   // the first index of this row
    uint64_t* list = nullptr;
    if constexpr (kBeam) {
        base = p.score[row];  // out_score may be the same array
        index0 = static_cast<uint32_t>(row % p.W) * p.V;
        list = p.lists + row * p.k;
        const bool ended = p.finished && __ldg(p.finished + row);
        if (bad_logit(base) || base == neg_inf() || ended) {  // no logits to read (the same branch in the whole cluster)
            sync(cluster, C);  // every CTA has read the score: the last beam to arrive may write over it
            if (rank != 0) return;
            for (int r = tid; r < p.k; r += kThreads) {
                uint64_t key = 0;
                if (r == 0) key = bad_logit(base) ? kFailed : base == neg_inf() ? 0 : key_of(base, index0 + p.eos);
                list[r] = key;
            }
            finish_beam(p, row, sh, turn, cluster);
            return;
        }
    }

    const Slice<kDtype> s(kBeam ? static_cast<const char*>(p.logits) + row / p.W * p.item_stride * Elem<kDtype>::kSize
                                : p.logits,
                          kBeam ? row % p.W : row, p.row_stride, p.V, rank, C);
    StreamedRow<kDtype, kThreads> x(s);

    // ---- one pass: the groups' maxima, the running maximum and sum of exp
    const float a = kLog2e * p.inv_t;
    static_assert(kBatch == StreamedRow<kDtype, kThreads>::kBatch, "a group is two threads' batches");
    Running run;
    float least = -neg_inf();  // of the groups' maxima above -inf
    const int groups = (s.count + kBatch * kThreads - 1) / (kBatch * kThreads) * kPairs;
    for (int g = tid; g < groups; g += kThreads) sh.group[g] = neg_inf();  // for warps past the slice's end
    __syncthreads();
    int batch = 0;
    x.each_batch([&](const uint4(&v)[kBatch], int) {
        const float t = vector_max<kDtype>(v);
        run.add<kDtype>(v, t, a);
        const float both = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
        if ((tid & 1) == 0) sh.group[batch * kPairs + tid / 2] = both;
        if (both > neg_inf()) least = fminf(least, both);
        ++batch;
    });
    if (x.edge_at >= 0) {
        run.add(x.edge, a);
        if (x.edge > neg_inf()) least = fminf(least, x.edge);
    }
    float m = warp_max(run.m);
    least = warp_min(least);
    if (lane == 0) {
        sh.red[0][warp] = m;
        sh.red[1][warp] = least;
    }
    __syncthreads();
    m = join_max(sh.red[0]);
    least = join_min(sh.red[1]);
    float sum = run.total(a) * ex2((run.m - m) * a);
    sum = warp_sum(sum);
    if (lane == 0) sh.red[2][warp] = sum;
    __syncthreads();
    sum = join_sum(sh.red[2]);
    if (tid == 0) {
        sh.part[0] = m;
        sh.part[1] = sum;
        sh.part[2] = least;
    }
    sync(cluster, C);
    float M = kLowest;
    for (int r = 0; r < C; ++r) {
        const float* q = cluster.map_shared_rank(sh.part, r);
        M = fmax_nan(M, q[0]);
        least = fminf(least, q[2]);
    }
    float S = 0.0f;
    for (int r = 0; r < C; ++r) {
        const float* q = cluster.map_shared_rank(sh.part, r);
        S += q[1] * ex2((q[0] - M) * a);
    }
    const float log_s = logf(S);
    const bool bad = S != S, empty = S == 0.0f;  // the same in the whole cluster

    // ---- the k best
    auto value = [&](float z) { return kBeam ? base + ((z - M) - log_s) : z; };
    int count = 0;
    if (!bad && !empty) {
        auto group_key = [&](float z) { return key_of(value(z), 0xFFFFFFFFu); };
        auto maxima = [&](auto f) {
            for (int g = tid; g < groups; g += kThreads) f(group_key(sh.group[g]));
            if (x.edge_at >= 0) f(group_key(x.edge));
        };
        auto entries = [&](auto f) {
            x.each([&](float z, int id) { f(key_of(value(z), index0 + id)); });
        };
        // the groups that reach the floor, a vector to a thread
        auto reached = [&](auto f) {
            const int n = static_cast<int>(min(sh.reached, static_cast<uint32_t>(kCap))) * (2 * kBatch);
            for (int i = tid; i < n; i += kThreads) {
                const int g = sh.reach[i / (2 * kBatch)], u = i / 2 % kBatch;
                const int j = (g / kPairs * kBatch + u) * kThreads + g % kPairs * 2 + i % 2;
                if (j >= s.count) continue;
                float z[P];
                unpack<kDtype>(ld_stream_v4(s.vec(j)), z);
#pragma unroll
                for (int e = 0; e < P; ++e) f(key_of(value(z[e]), index0 + s.elem0 + j * P + e));
            }
            if (x.edge_at >= 0) f(key_of(value(x.edge), index0 + x.edge_at));
        };
        const uint64_t lo = max(kFirstKey, group_key(least));
        const uint64_t hi = key_of(value(M), 0) + 1;
        // the maxima's keys have no index: their low halves, and the floor's, are zero
        uint64_t floor = max(kFirstKey, find_floor(maxima, p.k, p.k + p.k / 4 + 64, 32, lo, hi, sh, turn, cluster, C));
        for (int g = tid; g < groups; g += kThreads) {
            if (group_key(sh.group[g]) < floor) continue;
            const uint32_t at = atomicAdd(&sh.reached, 1u);
            if (at < kCap) sh.reach[at] = g;
        }
        __syncthreads();
        // more groups than the list holds have more entries than the buffer
        if (sh.reached > kCap && tid == 0) atom_add_cluster(cluster_addr(&sh.count, 0), kCap + 1u);
        count = gather(reached, floor, sh, cluster, C);
        if (count > kCap) {
            sync(cluster, C);
            if (rank == 0 && tid == 0) sh.count = 0;
            floor = max(kFirstKey, find_floor(entries, p.k, kCap, 0, kFirstKey, hi, sh, turn, cluster, C));
            count = gather(entries, floor, sh, cluster, C);
        }
    }
    sync(cluster, C);  // no CTA leaves while another reads its sums or its count
    if (rank != 0) return;

    if constexpr (kBeam) {
        for (int r = (bad ? 0 : count) + tid; r < p.k; r += kThreads) list[r] = bad && r == 0 ? kFailed : 0;
        if (!bad) rank_candidates(sh, count, p.k, [&](int r, uint64_t key) { list[r] = key; });
        finish_beam(p, row, sh, turn, cluster);
    } else {
        auto put = [&](int r, float v, int id) {
            const int64_t at = row * p.k + r;
            if constexpr (kDtype == kBF16)
                static_cast<uint16_t*>(p.values)[at] = static_cast<uint16_t>(__float_as_uint(v) >> 16);  // a copy
            else
                static_cast<float*>(p.values)[at] = v;
            p.index[at] = id;
        };
        for (int r = count + tid; r < p.k; r += kThreads) put(r, neg_inf(), -1);
        rank_candidates(sh, count, p.k, [&](int r, uint64_t key) {
            const uint32_t id = 0xFFFFFFFFu - static_cast<uint32_t>(key);
            float v = key_to_float(static_cast<uint32_t>(key >> 32));
            if (v == 0.0f) v = load_elem<kDtype>(s.row + static_cast<int64_t>(id) * Elem<kDtype>::kSize);  // -0 has 0's key
            put(r, v, id);
        });
        if (tid == 0) {
            p.lse[row] = bad ? quiet_nan() : empty ? neg_inf() : M * p.inv_t + log_s;
            p.status[row] = bad ? kReqNonfinite : empty ? kReqEmpty : kReqOk;
        }
    }
}

}  // namespace

cudaError_t launch_top_rows(const TopParams& p, cudaStream_t stream) {
    const int C = spread(p.N, p.V / (p.dtype == kBF16 ? 8 : 4), kThreads, kBatch * kBatches, kStreamFill);
    if (p.score)
        return p.dtype == kBF16 ? launch_row_kernel(top_kernel<kBF16, true>, p.N, C, kThreads, 0, stream, p)
                                : launch_row_kernel(top_kernel<kF32, true>, p.N, C, kThreads, 0, stream, p);
    return p.dtype == kBF16 ? launch_row_kernel(top_kernel<kBF16, false>, p.N, C, kThreads, 0, stream, p)
                            : launch_row_kernel(top_kernel<kF32, false>, p.N, C, kThreads, 0, stream, p);
}

}  // namespace dspark
