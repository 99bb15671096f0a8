// Rows of V logits split over the CTAs of a cluster, shared by the kernels of
// the kept top logits (top_rows.cu) and of their distillation (distill.cu):
// slices, running softmax sums, reductions and signals between warps and CTAs.
//
// A row may start at any element: the elements before its first 16-byte
// boundary and after its last whole vector (fewer than a vector each) are the
// row's edge, which rank 0 holds one element to a thread; the vectors between
// are dealt to the CTAs in contiguous slices.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace dspark {
namespace rows {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;

template <int kDtype>
struct Elem {
    static constexpr int kPer = kDtype == kBF16 ? 8 : 4;  // elements in a 16-byte vector
    static constexpr int kSize = kDtype == kBF16 ? 2 : 4;
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xFF800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7FC00000); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int kDtype>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[Elem<kDtype>::kPer]) {
    if constexpr (kDtype == kBF16) {
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
    } else {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
}

// Read-only loads that stay where they are written (the compiler may move an
// ordinary one down to its use, and its latency with it).
__device__ __forceinline__ uint32_t load_u32(const void* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float load_f32(const void* p) { return __uint_as_float(load_u32(p)); }
__device__ __forceinline__ uint32_t load_u16(const void* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float load_bf16(const void* p) { return __uint_as_float(load_u16(p) << 16); }
template <int kDtype>
__device__ __forceinline__ float load_elem(const char* p) {
    return kDtype == kBF16 ? load_bf16(p) : load_f32(p);
}

// One CTA's share of a row.
template <int kDtype>
struct Slice {
    const char* row;  // the row's first element
    int V;
    int head;         // elements before the first 16-byte boundary
    int tail0;        // first element after the last whole vector
    int elem0;        // element of this slice's first vector
    int count;        // vectors in this slice
    int rank;

    // C a power of two
    __device__ __forceinline__ Slice(const void* base, int64_t r, int64_t stride, int V_, int rank_, int C)
        : V(V_), rank(rank_) {
        constexpr int P = Elem<kDtype>::kPer, E = Elem<kDtype>::kSize;
        row = static_cast<const char*>(base) + r * stride * E;
        head = min(static_cast<int>((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / E, V);
        const int nvec = (V - head) / P;
        tail0 = head + nvec * P;
        const int per = (nvec + C - 1) >> (__ffs(C) - 1);
        const int first = min(rank * per, nvec);
        count = min(per, nvec - first);
        elem0 = head + first * P;
    }
    __device__ __forceinline__ const char* vec(int j) const {
        return row + static_cast<int64_t>(elem0) * Elem<kDtype>::kSize + static_cast<int64_t>(j) * 16;
    }
    // This thread's element of the row's edge, or -1 (rank 0: threads 0..7
    // hold the head, 32..39 the tail).
    __device__ __forceinline__ int edge_id() const {
        if (rank != 0) return -1;
        const int t = threadIdx.x;
        if (t < head) return t;
        if (t >= 32 && t - 32 < V - tail0) return tail0 + t - 32;
        return -1;
    }
    // The bit of element id in this slice's bitmap: kPer bits per vector, then
    // a word for the edge (head bits 0..7, tail bits 8..15).  -1: another CTA's.
    __device__ __forceinline__ int bit_of(int id) const {
        const int n = count * Elem<kDtype>::kPer;
        if (id >= elem0 && id < elem0 + n) return id - elem0;
        if (rank == 0 && id < head) return edge_word() * 32 + id;
        if (rank == 0 && id >= tail0) return edge_word() * 32 + 8 + id - tail0;
        return -1;
    }
    __device__ __forceinline__ int edge_word() const { return (count * Elem<kDtype>::kPer + 31) / 32; }
    __device__ __forceinline__ int bitmap_words() const { return edge_word() + 1; }
};

// Words of the largest bitmap a slice of a row of V elements needs.
__host__ __device__ inline int max_bitmap_words(int V, int C) { return (V / 4 + C - 1) / C * 4 / 32 + 4; }

// A vector whose elements marked in `bits` are -inf.
template <int kDtype>
__device__ __forceinline__ void drop_marked(uint4& v, uint32_t bits) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kDtype == kBF16) {
            if (bits >> (2 * i) & 1u) w[i] = (w[i] & 0xFFFF0000u) | 0xFF80u;
            if (bits >> (2 * i + 1) & 1u) w[i] = (w[i] & 0xFFFFu) | 0xFF800000u;
        } else {
            if (bits >> i & 1u) w[i] = 0xFF800000u;
        }
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
}
template <int kDtype>
__device__ __forceinline__ uint4 neg_inf_vector() {
    const uint32_t w = kDtype == kBF16 ? 0xFF80FF80u : 0xFF800000u;
    return make_uint4(w, w, w, w);
}

// Two 32-bit values in one register pair, for the paired arithmetic.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split(uint64_t p, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The largest element of n vectors (a NaN may be passed over).
template <int kDtype, int n>
__device__ __forceinline__ float vector_max(const uint4 (&v)[n]) {
    if constexpr (kDtype == kBF16) {
        __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&v[0].x);
#pragma unroll
        for (int u = 0; u < n; ++u) {
            const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v[u]);
            m = __hmax2(__hmax2(m, __hmax2(w[0], w[1])), __hmax2(w[2], w[3]));
        }
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        float m = neg_inf();
#pragma unroll
        for (int u = 0; u < n; ++u)
            m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(v[u].x), __uint_as_float(v[u].y))),
                      fmaxf(__uint_as_float(v[u].z), __uint_as_float(v[u].w)));
        return m;
    }
}
// f(i, p): the vector's elements 2 i and 2 i + 1 as a pair.
template <int kDtype, class F>
__device__ __forceinline__ void each_pair(const uint4& v, F f) {
    if constexpr (kDtype == kBF16) {
        f(0, pair(bf16_lo(v.x), bf16_hi(v.x)));
        f(1, pair(bf16_lo(v.y), bf16_hi(v.y)));
        f(2, pair(bf16_lo(v.z), bf16_hi(v.z)));
        f(3, pair(bf16_lo(v.w), bf16_hi(v.w)));
    } else {
        f(0, pair(__uint_as_float(v.x), __uint_as_float(v.y)));
        f(1, pair(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
}

// A product that is rounded by itself (never contracted into an addition).
__device__ __forceinline__ float product(float x, float y) {
    float r;
    asm("mul.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// exp2((x - m) a) as one fused multiply-add and an exp2: x a - fl(m a).  What the
// rounding of m a scales all values by, remainder(m, a), is left to the caller.
// Where |m a| passes 2^29 (rows of a type's lowest value) neighbouring values of
// x differ by 32 and more after scaling, so that only those equal to m count: a
// smaller factor that takes m to 2^29 says the same and overflows nowhere.
constexpr float kFarthest = 536870912.0f;
struct Scale {
    float a, shift;  // x a + shift
    __device__ __forceinline__ Scale(float m, float a_) : a(a_), shift(-product(m, a_)) {
        if (!(fabsf(shift) < kFarthest)) {
            a = kFarthest / fabsf(m);
            shift = -product(m, a);
        }
    }
    __device__ __forceinline__ float exp_of(float x) const { return ex2(fmaf(x, a, shift)); }
    // 1 / exp_of(m)
    __device__ __forceinline__ float remainder(float m) const { return ex2(-fmaf(m, a, shift)); }
};
template <int kDtype, int n, class F>
__device__ __forceinline__ void each_exp(const uint4 (&v)[n], const Scale& s, F f) {
    const uint64_t aa = pair(s.a, s.a), shift = pair(s.shift, s.shift);
    float x, y;
#pragma unroll
    for (int u = 0; u < n; ++u)
        each_pair<kDtype>(v[u], [&](int i, uint64_t p) {
            split(fma2(p, aa, shift), x, y);
            f(u, i, pair(ex2(x), ex2(y)));
        });
}

// The running maximum m of a thread's elements and the sum of exp2((x - m) a);
// m starts at the lowest finite value, so that -inf contributes exp2(-inf) = 0.
// NaN and +inf make the sum NaN.
struct Running {
    float m = kLowest;
    uint64_t sum = 0;  // two partial sums, still to be multiplied by Scale(m, a).remainder(m)
    __device__ __forceinline__ void raise(float top, float a) {
        if (top > m) {
            const float ma = product(m, a), to = product(top, a);
            const float f = fabsf(ma) < kFarthest && fabsf(to) < kFarthest ? ex2(ma - to) : 0.0f;
            sum = mul2(sum, pair(f, f));
            m = top;
        }
    }
    template <int kDtype, int n>
    __device__ __forceinline__ void add(const uint4 (&v)[n], float top, float a) {
        raise(top, a);
        each_exp<kDtype>(v, Scale(m, a), [&](int, int, uint64_t e) { sum = add2(sum, e); });
    }
    __device__ __forceinline__ void add(float x, float a) {
        raise(x, a);
        sum = add2(sum, pair(Scale(m, a).exp_of(x), 0.0f));
    }
    __device__ __forceinline__ float total(float a) const {
        float x, y;
        split(sum, x, y);
        return (x + y) * Scale(m, a).remainder(m);
    }
};

// The values of one CTA's share of a row.  Elements whose bit is set in the
// bitmap given to set_drop (shared memory) read as -inf.  A streamed row is
// read from memory again by every pass over it.
template <int kDtype, int kThreads>
struct StreamedRow {
    static constexpr int P = Elem<kDtype>::kPer;
    static constexpr int kBatch = 4;  // vectors in flight per thread
    const Slice<kDtype>& s;
    const uint32_t* drop = nullptr;
    int edge_at;
    float edge;

    __device__ __forceinline__ explicit StreamedRow(const Slice<kDtype>& slice) : s(slice) {
        edge_at = s.edge_id();
        edge = edge_at >= 0 ? load_elem<kDtype>(s.row + static_cast<int64_t>(edge_at) * Elem<kDtype>::kSize)
                            : neg_inf();
    }
    __device__ __forceinline__ void set_drop(const uint32_t* bits) {
        drop = bits;
        const int b = edge_at >= 0 ? s.bit_of(edge_at) : -1;
        if (b >= 0 && (bits[b >> 5] >> (b & 31) & 1u)) edge = neg_inf();
    }
    // f(v, j0): vectors j0, j0 + kThreads, ... of the slice, -inf past its end.
    // A warp's lanes make the same number of calls.
    template <class F>
    __device__ __forceinline__ void each_batch(F f) const {
        for (int j0 = threadIdx.x; (j0 & ~31) < s.count; j0 += kBatch * kThreads) {
            uint4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                v[u] = j0 + u * kThreads < s.count ? ld_stream_v4(s.vec(j0 + u * kThreads)) : neg_inf_vector<kDtype>();
            if (drop) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int b = (j0 + u * kThreads) * P;
                    const uint32_t bits = j0 + u * kThreads < s.count ? drop[b >> 5] >> (b & 31) & ((1u << P) - 1u) : 0u;
                    if (bits) drop_marked<kDtype>(v[u], bits);
                }
            }
            f(v, j0);
        }
    }
    // f(x, id) for every element this thread reads
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        each_batch([&](const uint4(&v)[kBatch], int j0) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (j0 + u * kThreads >= s.count) break;
                float x[P];
                unpack<kDtype>(v[u], x);
#pragma unroll
                for (int i = 0; i < P; ++i) f(x[i], s.elem0 + (j0 + u * kThreads) * P + i);
            }
        });
        if (edge_at >= 0) f(edge, edge_at);
    }
    // the running maximum and sum of exp2 over this thread's elements
    __device__ __forceinline__ Running running(float a) const {
        Running r;
        each_batch([&](const uint4(&v)[kBatch], int) { r.add<kDtype>(v, vector_max<kDtype>(v), a); });
        if (edge_at >= 0) r.add(edge, a);
        return r;
    }
};

// ------------------------------------------------------------- reductions
// The largest and the least value of a warp (a NaN is passed over).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_min(float v) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
template <int kLanes = 32, class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// The reduction of one value per warp, in shared memory behind a barrier, in
// every lane of the calling warp.
template <int kWarps>
__device__ __forceinline__ float join_max(const float (&w)[kWarps]) {
    return warp_max((threadIdx.x & 31) < kWarps ? w[threadIdx.x & 31] : neg_inf());
}
template <int kWarps>
__device__ __forceinline__ float join_min(const float (&w)[kWarps]) {
    return warp_min((threadIdx.x & 31) < kWarps ? w[threadIdx.x & 31] : -neg_inf());
}
template <class T, int kWarps>
__device__ __forceinline__ T join_sum(const T (&w)[kWarps]) {
    return warp_sum((threadIdx.x & 31) < kWarps ? w[threadIdx.x & 31] : T(0));
}
// A warp's maximum and its sum of exp2 against it, from its first kLanes lanes'
// pairs (the sum in those lanes only).
template <int kLanes = 32>
__device__ __forceinline__ void join_lanes(float& m, float& sum, float a) {
    const float top = warp_max(m);
    sum = warp_sum<kLanes>(sum * ex2((m - top) * a));
    m = top;
}
// The same from one pair per warp.
template <int kWarps>
__device__ __forceinline__ void join_warps(const float (&w)[kWarps], const float (&part)[kWarps], float a, float& m,
                                           float& sum) {
    const int lane = threadIdx.x & 31;
    m = lane < kWarps ? w[lane] : kLowest;
    sum = lane < kWarps ? part[lane] : 0.0f;
    join_lanes(m, sum, a);
}

// --------------------------------------------------- signals between warps
// Named barriers of n threads: the arriving side does not wait; what it wrote
// before is seen by the side that does.
__device__ __forceinline__ void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// The address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t atom_add_cluster(uint32_t addr, uint32_t v) {
    uint32_t old;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// Stores to another CTA's shared memory that complete their bytes on its mbarrier.
__device__ __forceinline__ void push_v4(uint32_t dst, float x, float y, float z, float w, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(__float_as_uint(z)), "r"(__float_as_uint(w)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void push_u32(uint32_t dst, uint32_t x, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst), "r"(x), "r"(bar)
                 : "memory");
}
// mbar_wait for data that other CTAs of the cluster stored.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (t0 == 0)
            t0 = globaltimer_ns();
        else if (globaltimer_ns() - t0 > limit_ns)
            return false;
    }
}

__device__ __forceinline__ void sync(const cg::cluster_group& cluster, int C) {
    if (C == 1)
        __syncthreads();
    else
        cluster.sync();
}

}  // namespace rows

constexpr int kSms = 152;
constexpr int kStreamFill = 2 * kSms;

// CTAs to a row: enough that a thread has at most `most` vectors of it, and, while
// there are few CTAs (n C <= fill), more of them up to eight: a row then takes less
// time, but joining its parts more.  Streamed kernels take fill = kStreamFill = 304, measured
// against 152, 608 and 1,216 (device us): selection of 32 x 8 beams 23.5 against
// 25.2, 30.4 and 41.6; loss of 300 rows 23.5 against 26.3, 28.4 and 32.2; rows by
// the thousand the same at all but the last.
inline int spread(int64_t n, int64_t vectors, int threads, int most, int fill) {
    int C = 1;
    while (C < rows::kMaxCluster && (vectors > static_cast<int64_t>(C) * most * threads ||
                                     (n * C <= fill && vectors > static_cast<int64_t>(C) * threads)))
        C *= 2;
    return C;
}

// Launch of `kernel` on clusters of C CTAs.
template <class... Params, class... Args>
inline cudaError_t launch_row_kernel(void (*kernel)(Params...), int64_t clusters, int C, int threads, size_t smem,
                                     cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * C));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dspark
