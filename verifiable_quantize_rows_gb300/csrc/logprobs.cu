// logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of logits, and their gradient.
//
//   lse = m + log S,  S = sum_j e_j,  e_j = exp(x_j - m),  m = max_j x_j;
//   entropy = log S - A / S,  A = sum_j e_j (x_j - m);
//   dx_j = g_lp ([j = t] - p_j) - g_H p_j (x_j - lse + H).
//
// Forward: one read of the logits, which is what bounds it (HBM).  Each thread
// keeps a running maximum with S and A = sum e (x - m) relative to it; a new
// maximum m' scales S by f = e^(m - m') and makes A f (A + (m - m') S).
//
// The top alternatives come from the same read.  Of the threads' maxima so far, the
// n-th largest of each warp's 32 and of those the least over W warps has W n
// values at least as large: what is not above it cannot be among the top W n.
// What is goes to a list in shared memory, a few hundred entries a row, from which
// the best 32 are sorted out at the end.  Entries are 64-bit keys, the value's order
// above the complement of the index, so that of equals the lowest index is the
// largest key.  Rounds go up in index, so after the first an equal value is never
// better.  Where the list overflows (logits that keep rising), a second read in
// steps of one round sorts it whenever it is full.
//
// Measured: 8192 x 50304 f32 236 us without the top (the floor's own rate), 257 with the
// top 1, 295 with the top 20 (0.83 of it); bf16 187 and 344; 1 f32 row with the top 5 7.8.
// What bounds it: HBM without the top; with it the least's barriers, the branches that list
// an entry and a row's last sort, while which a CTA reads nothing; one row the launch,
// a cluster's start and its barriers.  (Listing a thread's candidates by one atomic
// addition from a mask of its 16: 348 us.  The least after every round up to 4, and at
// twice as many after: 307.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "serve.cuh"

namespace cg = cooperative_groups;

namespace bsg {
namespace {

constexpr int kRound = 16;        // elements of a thread in a round
constexpr int kGradThreads = 256;
// Entries that fit the list of a CTA: a round's, and some.
__host__ __device__ constexpr int list_size(int threads) { return threads * kRound + 512; }
constexpr int kMaxRanks = 16;     // CTAs of a row
constexpr float kLog2e = 1.4426950408889634f;

// The 16-byte vectors that cover a row: vector v holds elements
// [v kPer - off, (v + 1) kPer - off) of it, off the row's distance from 16 bytes.
template <typename T>
struct RowVectors {
    static constexpr int kPer = 16 / sizeof(T);
    const T *row;
    int64_t V, count;
    int off;
    __device__ RowVectors(const T *r, int64_t n) : row(r), V(n) {
        off = (int)(reinterpret_cast<uintptr_t>(r) % 16 / sizeof(T));
        count = (n + off + kPer - 1) / kPer;
    }
    static __device__ __forceinline__ void load_whole(const T *at, float (&x)[kPer]) {
        uint4 w;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "l"(at));
        const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = to_f32(e[i]);
    }
    // Elements of vector v, -inf outside the row.
    __device__ __forceinline__ void load(int64_t v, float (&x)[kPer]) const {
        const int64_t j0 = v * kPer - off;
        if (j0 >= 0 && j0 + kPer <= V) {
            load_whole(row + j0, x);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                x[i] = j0 + i >= 0 && j0 + i < V ? to_f32(row[j0 + i]) : -INFINITY;
        }
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Largest of the three, NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Running maximum, S and A / ln 2, of a thread or of several joined.
struct Sums {
    float m = -INFINITY, s = 0.0f, a = 0.0f;
    // Relative to another maximum, not below this one.
    __device__ __forceinline__ void raise(float to) {
        if (m == -INFINITY || to == m) {  // nothing yet (s = a = 0), or nothing to do
            m = to;
            return;
        }
        const float y = fmaxf((m - to) * kLog2e, -1e4f), f = ex2(y);  // 2^-1e4 is 0
        a = f * fmaf(y, s, a);
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void join(Sums o) {
        const float to = fmaxf(m, o.m);
        raise(to);
        o.raise(to);
        s += o.s, a += o.a;
    }
};

// Values in order as unsigned numbers, -0 as +0; none is 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t v) {
    return __uint_as_float(v & 0x80000000u ? v & 0x7fffffffu : ~v);
}
// A value and its index as a key: larger is better.  No valid key is 0.
__device__ __forceinline__ uint64_t key_of(float x, int64_t j) {
    return (uint64_t)ordered(x) << 32 | (uint32_t)~(uint32_t)j;
}
__device__ __forceinline__ float key_value(uint64_t k) { return value_of((uint32_t)(k >> 32)); }
__device__ __forceinline__ int32_t key_index(uint64_t k) { return (int32_t)~(uint32_t)k; }

// One step of a bitonic network over a warp, larger keys first where `down`.
__device__ __forceinline__ uint64_t exchange(uint64_t k, int distance, bool down) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, k, distance);
    const bool low = (threadIdx.x & distance) == 0;
    return (k > o) == (low == down) ? k : o;
}
__device__ __forceinline__ uint64_t warp_sort(uint64_t k) {  // descending
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int d = size / 2; d; d /= 2) k = exchange(k, d, size == 32 || (lane & size) == 0);
    return k;
}
// The best 32 of two descending lists, descending.
__device__ __forceinline__ uint64_t warp_merge(uint64_t k, uint64_t o) {
    const uint64_t r = __shfl_sync(0xffffffffu, o, 31 - threadIdx.x % 32);
    k = k > r ? k : r;
#pragma unroll
    for (int d = 16; d; d /= 2) k = exchange(k, d, true);
    return k;
}

// The best 32 of the warps' descending lists, in warp 0.
template <int kWarps>
__device__ __forceinline__ uint64_t join_warps(uint64_t best, uint64_t (*lists)[32]) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int half = kWarps / 2; half; half /= 2) {
        if (warp >= half && warp < 2 * half) lists[warp][lane] = best;
        __syncthreads();
        if (warp < half) best = warp_merge(best, lists[warp + half][lane]);
    }
    return best;
}

// Sorts the best 32 of list[0..n) to its front, by all threads; unused places 0.
template <int kWarps>
__device__ void sort_list(uint64_t *list, int n, uint64_t (*lists)[32]) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t best = 0;
    for (int b = warp * 32; b < n; b += kWarps * 32) {
        uint64_t k = b + lane < n ? list[b + lane] : 0;
        if (!__any_sync(0xffffffffu, k > __shfl_sync(0xffffffffu, best, 31))) continue;
        best = warp_merge(best, warp_sort(k));
    }
    best = join_warps<kWarps>(best, lists);
    if (warp == 0) list[lane] = best;
    __syncthreads();
}

struct LogprobsArgs {
    const int64_t *target;
    float *logprob, *entropy, *lse, *top_logprob;
    int32_t *top_id, *dstatus;
    int64_t V, ldl;
    int top;
};

// A cluster of CTAs to a row (or one CTA), each a contiguous share of its vectors.
template <typename T, bool kTop, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    logprobs_kernel(const T *__restrict__ logits, const __grid_constant__ LogprobsArgs a) {
    constexpr int kPer = RowVectors<T>::kPer, kVec = kRound / kPer;
    constexpr int kLpWarps = kThreads / 32, kList = list_size(kThreads);
    __shared__ uint64_t list[kTop ? kList : 1];
    __shared__ uint64_t lists[kTop ? kLpWarps : 1][32];
    __shared__ float warp_least[kLpWarps];
    __shared__ Sums warp_sums[kLpWarps];
    __shared__ Sums cta_sums;
    __shared__ int listed;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int64_t r = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const RowVectors<T> row(logits + r * a.ldl, a.V);
    const int64_t v0 = row.count * rank / ranks, v1 = row.count * (rank + 1) / ranks;
    if (tid == 0) listed = 0;
    if (kTop) __syncthreads();

    Sums sums;
    bool bad = false;
    float least = -INFINITY;  // what is not above it is not among the top
    // Lists what is not `<= above` (NaN: everything).  True where the list has less
    // than a round's room left, or none.
    auto push = [&](float (&x)[kVec][kPer], int64_t v, float above) {
        bool full = false;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            float most = x[i][0];
#pragma unroll
            for (int e = 1; e < kPer; ++e) most = fmaxf(most, x[i][e]);
            if (most <= above) continue;
            const int64_t j0 = (v + i * kThreads) * kPer - row.off;
            // its first element of the row, and how many there are
            const int lo = j0 < 0 ? (int)-j0 : 0;
            const uint32_t in = v + i * kThreads < v1 ? (uint32_t)((a.V - j0 < kPer ? (int)(a.V - j0) : kPer) - lo) : 0;
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (!(x[i][e] <= above) && (uint32_t)(e - lo) < in) {
                    const int at = atomicAdd(&listed, 1);
                    if (at < kList) list[at] = key_of(x[i][e], j0 + e);
                    full |= at >= kList - kThreads * kRound - 1;
                }
        }
        return full;
    };
    // The least that `top` of the values read so far reach: of each warp's maxima the
    // n-th largest, n kLpWarps >= top, and of those the smallest.  All threads together.
    auto find_least = [&]() {
        uint32_t mine = ordered(sums.m), nth = 0;
        for (int k = 0; k < a.top; k += kLpWarps) {
            nth = __reduce_max_sync(0xffffffffu, mine);
            const uint32_t has = __ballot_sync(0xffffffffu, mine == nth);
            if (lane == __ffs(has) - 1) mine = 0;
        }
        __syncthreads();  // the last one's have been read
        if (lane == 0) warp_least[warp] = value_of(nth);
        __syncthreads();
        float l = warp_least[0];
#pragma unroll
        for (int w = 1; w < kLpWarps; ++w) l = fminf(l, warp_least[w]);
        least = fmaxf(least, l);
    };
    // Just below x, so that x itself is above it.
    auto below = [](float x) {
        const uint32_t b = __float_as_uint(x + 0.0f);
        return x == -INFINITY ? NAN : b == 0 ? -1.4e-45f : __uint_as_float(b & 0x80000000u ? b + 1 : b - 1);
    };
    auto load = [&](float (&x)[kVec][kPer], int64_t v) {
        const int64_t base = v - tid, j0 = base * kPer - row.off;  // the round's, of all threads
        if (j0 >= 0 && j0 + kThreads * kRound <= a.V && base + kVec * kThreads <= v1) {
            const T *at = row.row + j0 + tid * kPer;
#pragma unroll
            for (int i = 0; i < kVec; ++i) RowVectors<T>::load_whole(at + i * kThreads * kPer, x[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if (v + i * kThreads < v1)
                row.load(v + i * kThreads, x[i]);
            else
#pragma unroll
                for (int e = 0; e < kPer; ++e) x[i][e] = -INFINITY;
        }
    };
    float x[kVec][kPer], next[kVec][kPer];
    load(next, v0 + tid);
    int round = 0;
    for (int64_t v = v0 + tid; v - tid < v1; v += kVec * kThreads, ++round) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[i][e] = next[i][e];
        load(next, v + kVec * kThreads);
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int e = 0; e < kPer; e += 2) most = max_nan(most, x[i][e], x[i][e + 1]);
        bad |= !(most < INFINITY);
        if (most > sums.m) sums.raise(most);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                // -inf, and -inf less -inf, count as far below: 0 in both sums
                const float y = fmaxf((x[i][e] - sums.m) * kLog2e, -1e4f), p = ex2(y);
                sums.s += p;
                sums.a = fmaf(p, y, sums.a);
            }
        if (kTop) {
            // after 1, 2, 4, 8 ... rounds; what equals the least of this round counts
            const bool due = (round & (round + 1)) == 0;
            if (due) find_least();
            const float above = due ? below(least) : least;
            if (!(most <= above)) push(x, v, above);
        }
    }
    if (kTop && __syncthreads_or(listed > kList)) {
        // the list has overflowed: again, round by round
        __syncthreads();
        if (tid == 0) listed = 0;
        least = -INFINITY;
        __syncthreads();
        for (int64_t v = v0 + tid; v - tid < v1; v += kVec * kThreads) {
            load(x, v);
            if (__syncthreads_or(push(x, v, v - tid == v0 ? NAN : least))) {
                sort_list<kLpWarps>(list, listed, lists);
                if (list[31]) least = key_value(list[31]);
                if (tid == 0) listed = 32;
                __syncthreads();
            }
        }
    }
    if (bad) set_status(a.dstatus, BSG_DSTATUS_NONFINITE);

    // Join the threads, the warps and the cluster, in that order.
    auto join_lanes = [](Sums x) {  // of all lanes, in each
#pragma unroll
        for (int o = 16; o; o /= 2) {
            Sums other;
            other.m = __shfl_xor_sync(0xffffffffu, x.m, o);
            other.s = __shfl_xor_sync(0xffffffffu, x.s, o);
            other.a = __shfl_xor_sync(0xffffffffu, x.a, o);
            x.join(other);
        }
        return x;
    };
    sums = join_lanes(sums);
    if (lane == 0) warp_sums[warp] = sums;
    __syncthreads();
    if (kTop) sort_list<kLpWarps>(list, listed, lists);
    Sums all;
    if (warp == 0) all = join_lanes(lane < kLpWarps ? warp_sums[lane] : Sums());
    if (ranks > 1) {
        if (tid == 0) cta_sums = all;
        cluster.sync();
        if (rank == 0) {
            if (kTop) {  // a few CTAs' lists to a warp, all on their way at once
                constexpr int kEach = kMaxRanks / kLpWarps;
                uint64_t best = 0, more[kEach];
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    more[i] = warp + i * kLpWarps < ranks ? cluster.map_shared_rank(list, warp + i * kLpWarps)[lane] : 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) best = warp_merge(best, more[i]);
                best = join_warps<kLpWarps>(best, lists);
                if (warp == 0) list[lane] = best;  // warp 0 has read its own
            }
            all = join_lanes(lane < ranks ? *cluster.map_shared_rank(&cta_sums, lane) : Sums());
        }
        cluster.sync();  // no CTA leaves while its results are read
        if (rank > 0) return;
    }
    if (warp > 0) return;

    const bool none = all.m == -INFINITY;  // every logit is -inf
    const float log_s = none ? 0.0f : logf(all.s);
    if (lane == 0) {
        if (a.lse) a.lse[r] = all.m + log_s;
        if (a.entropy) a.entropy[r] = none ? 0.0f : log_s - all.a * 0.69314718055994531f / all.s;
        const int64_t g = a.target ? a.target[r] : -1;
        if (g >= a.V) set_status(a.dstatus, BSG_DSTATUS_RANGE);
        if (a.logprob)
            a.logprob[r] = g < 0        ? 0.0f
                           : g >= a.V   ? NAN
                           : none       ? -INFINITY
                                        : to_f32(row.row[g]) - all.m - log_s;
    }
    if (kTop && lane < a.top) {
        const uint64_t k = list[lane];
        a.top_logprob[r * a.top + lane] = none ? -INFINITY : key_value(k) - all.m - log_s;
        a.top_id[r * a.top + lane] = key_index(k);
    }
}

// ---- gradient -----------------------------------------------------------------
//
// One read and one write of every element, four 16-byte vectors to a thread, all read
// before the first is written.  HBM bounds it: 8192 x 50304 f32 478 us, the floor's
// own rate (0.83 of the peak, reads and writes together); 97 x 12289 bf16 4.5 us, a
// launch.
constexpr int kGradVec = 4;  // vectors of a thread

template <typename T>
__global__ void __launch_bounds__(kGradThreads)
    logprobs_backward_kernel(const T *logits, int64_t V, int64_t ldl,
                             const int64_t *__restrict__ target, const float *__restrict__ lse,
                             const float *__restrict__ entropy,
                             const float *__restrict__ g_logprob,
                             const float *__restrict__ g_entropy, T *dlogits, int64_t ldd,
                             int blocks, int32_t *__restrict__ dstatus) {
    constexpr int kPer = 16 / sizeof(T);
    const int64_t r = blockIdx.x / blocks;
    const T *x = logits + r * ldl;
    T *dx = dlogits + r * ldd;
    const int64_t t = target ? target[r] : -1;
    const float L = lse[r], H = g_entropy ? entropy[r] : 0.0f;
    const float gl = g_logprob && t >= 0 ? g_logprob[r] : 0.0f;
    const float gh = g_entropy ? g_entropy[r] : 0.0f;
    const bool bad_target = t >= V;
    if (bad_target && threadIdx.x == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
    // vectors by the logits' alignment; the gradient's may be another
    const int off = (int)(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    const bool same = reinterpret_cast<uintptr_t>(dx) % 16 == reinterpret_cast<uintptr_t>(x) % 16;
    const int64_t j_first = ((int64_t)(blockIdx.x % blocks) * kGradVec * kGradThreads + threadIdx.x) * kPer - off;
    bool bad = false;
    auto gradient = [&](float v, int64_t j) {
        bad |= !(v < INFINITY);
        const float lp = v - L, p = ex2(lp * kLog2e);
        float d = p > 0.0f ? -p * fmaf(gh, lp + H, gl) : 0.0f;
        if (j == t) d += gl;
        if (L == -INFINITY) d = 0.0f;
        return bad_target ? NAN : d;
    };
    uint4 w[kGradVec];
#pragma unroll
    for (int i = 0; i < kGradVec; ++i) {
        const int64_t j = j_first + (int64_t)i * kGradThreads * kPer;
        // not the read-only path: the gradient may take the logits' place
        if (j >= 0 && j + kPer <= V)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                         : "l"(x + j)
                         : "memory");
    }
#pragma unroll
    for (int i = 0; i < kGradVec; ++i) {
        const int64_t j = j_first + (int64_t)i * kGradThreads * kPer;
        if (j >= 0 && j + kPer <= V) {
            T *e = reinterpret_cast<T *>(&w[i]);
#pragma unroll
            for (int k = 0; k < kPer; ++k) e[k] = from_f32<T>(gradient(to_f32(e[k]), j + k));
            if (same)
                __stcs(reinterpret_cast<uint4 *>(dx + j), w[i]);
            else
#pragma unroll
                for (int k = 0; k < kPer; ++k) dx[j + k] = e[k];
        } else {
            for (int k = 0; k < kPer; ++k)
                if (j + k >= 0 && j + k < V) dx[j + k] = from_f32<T>(gradient(to_f32(x[j + k]), j + k));
        }
    }
    if (bad) set_status(dstatus, BSG_DSTATUS_NONFINITE);
}

template <typename T, bool kTop, int kThreads>
cudaError_t launch_forward(const T *logits, const LogprobsArgs &a, int64_t M, int ranks, cudaStream_t st) {
    auto *kernel = logprobs_kernel<T, kTop, kThreads>;
    static bool set[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        set[dev] = true;
    }
    if (M * ranks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(M * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, logits, a);
}

// A row to one CTA of 128 threads where there are rows for every SM (256: 349 against
// 297 us at 8192 x 50304, since a row's sorting and joining are per warp), else
// to a cluster of 256-thread ones, with a round for each of them at least.
template <typename T, bool kTop>
cudaError_t launch_rows(const T *logits, const LogprobsArgs &a, int64_t M, cudaStream_t st) {
    int ranks = 1;
    while (ranks < kMaxRanks && M * ranks < device_sm_count() && a.V > (int64_t)ranks * 256 * kRound) ranks *= 2;
    return ranks == 1 && M >= device_sm_count() ? launch_forward<T, kTop, 128>(logits, a, M, 1, st)
                                                : launch_forward<T, kTop, 256>(logits, a, M, ranks, st);
}

}  // namespace

cudaError_t launch_logprobs(const void *logits, int dtype, int64_t M, int64_t V, int64_t ldl,
                            const int64_t *target, int top, float *logprob, float *entropy,
                            float *lse, float *top_logprob, int32_t *top_id, int32_t *dstatus,
                            cudaStream_t st) {
    const LogprobsArgs a{target, logprob, entropy, lse, top_logprob, top_id, dstatus, V, ldl, top};
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const T *x = static_cast<const T *>(logits);
        return top ? launch_rows<T, true>(x, a, M, st) : launch_rows<T, false>(x, a, M, st);
    });
}

cudaError_t launch_logprobs_backward(const void *logits, int dtype, int64_t M, int64_t V,
                                     int64_t ldl, const int64_t *target, const float *lse,
                                     const float *entropy, const float *g_logprob,
                                     const float *g_entropy, void *dlogits, int64_t ldd,
                                     int32_t *dstatus, cudaStream_t st) {
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t per = kGradVec * kGradThreads * (16 / (int64_t)sizeof(T));
        const int64_t blocks = (V + 16 / (int64_t)sizeof(T) - 1 + per - 1) / per;  // with a shifted start
        if (M > INT32_MAX / blocks) return cudaErrorInvalidValue;
        logprobs_backward_kernel<T><<<(unsigned)(M * blocks), kGradThreads, 0, st>>>(
            static_cast<const T *>(logits), V, ldl, target, lse, entropy, g_logprob, g_entropy,
            static_cast<T *>(dlogits), ldd, (int)blocks, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace bsg
