// kv8_more.cu -- attention over the int8 cache for any number of query tokens through a
// window with sinks, and behind a prefix that all sequences share: how a call is cut into
// chunks, its launches, and the join of the chunks.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bsg_ptx.cuh"
#include "kv8_more.h"
#include "serve.cuh"

namespace bsg {
namespace {

// ---- the join ---------------------------------------------------------------
//
// A row's output from the partial ones of one or two lists of chunks (its own positions',
// and the prefix's): each relative to its own reference, in units of log 2.  A chunk whose
// sum is 0 saw nothing, and its output is not read.  A CTA to a row: it waits for its loads, twice
// (weights, then outputs); by itself, caches cold, 13 us for 2048 rows of 128 dims behind 19 shared
// chunks and their own, 5 for 48 rows of 64.
struct JoinArgs {
    bsg_tokens out;
    int kv_heads, heads, tokens, B;
    const int32_t *lens, *counts;  // counts: window; lens: shared, whose idle rows give 0
    int64_t most;                  // positions of a table
    const float *o[2];
    const float2 *ml[2];
    int splits[2];                 // of [0]: own chunks, [sequence][head][token, head of the group][split]; [1]: the
    float *lse;                    // prefix's, [head][sequence, token, head of the group][split], or 0
};

constexpr int kJoinThreads = 128;
constexpr int kMaxChunks = 2048;  // of both lists: no plan has more than 1024 to a list

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_lists_kernel(const __grid_constant__ JoinArgs a) {
    constexpr int kCols = D / 4, kSides = kJoinThreads / kCols;
    __shared__ float4 o_s[kSides][kCols];
    const int share = a.heads / a.kv_heads, tid = threadIdx.x;
    const int h = blockIdx.x % a.heads, t = blockIdx.x / a.heads % a.tokens, b = blockIdx.x / a.heads / a.tokens;
    const int hk = h / share;
    bool idle = false;
    griddep_wait();  // every block, those of tokens that are not there too: this grid never ends before the ones it joins
    if (a.counts) {
        const int count = __ldg(a.counts + b);
        if (t >= count || count > a.tokens) return;
    }
    if (a.lens) {
        int64_t len = __ldg(a.lens + b);
        idle = min(len, a.most) - a.tokens + t < 0;
    }
    const int64_t row[2] = {((int64_t)b * a.kv_heads + hk) * a.tokens * share + t * share + h % share,
                            (((int64_t)hk * a.B + b) * a.tokens + t) * share + h % share};
    const int n = a.splits[0] + a.splits[1];
    auto at = [&](int i) {  // chunk i: its list's place
        return i < a.splits[0] ? row[0] * a.splits[0] + i : row[1] * a.splits[1] + i - a.splits[0];
    };
    // the chunks' weights first, a thread each, so that the outputs' loads wait for nothing
    __shared__ float f_s[kMaxChunks], red[kJoinThreads / 32];
    float m = -3.0e38f, l = 0.0f;
    if (!idle)
        for (int i = tid; i < n; i += kJoinThreads) {
            const float2 x = a.ml[i >= a.splits[0]][at(i)];
            if (x.y != 0.0f) m = fmaxf(m, x.x);
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (tid % 32 == 0) red[tid / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) m = fmaxf(m, red[i]);
    __syncthreads();
    for (int i = tid; i < n; i += kJoinThreads) {
        const float2 x = a.ml[i >= a.splits[0]][at(i)];
        const float f = x.y == 0.0f || idle ? 0.0f : exp2_of(x.x - m);
        f_s[i] = f;
        if (f != 0.0f) l = fmaf(x.y, f, l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (tid % 32 == 0) red[tid / 32] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) l += red[i];
    const int col = tid % kCols, side = tid / kCols;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (side < kSides)
#pragma unroll 4
        for (int i = side; i < n; i += kSides) {
            const float f = f_s[i];
            if (f == 0.0f) continue;  // what a chunk that saw nothing left is no output
            const float4 v = *reinterpret_cast<const float4 *>(a.o[i >= a.splits[0]] + at(i) * D + 4 * col);
            o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
        }
    if (side < kSides) o_s[side][col] = o;
    __syncthreads();
    const bool some = l > 0.0f || l != l;
    const float inv = some ? 1.0f / l : 0.0f;
    T *out = static_cast<T *>(a.out.data) + b * a.out.stride_batch + t * a.out.stride_token + h * a.out.stride_head;
    for (int d = tid; d < D; d += kJoinThreads) {
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < kSides; ++i) y += reinterpret_cast<const float *>(&o_s[i][d / 4])[d % 4];
        out[d] = from_f32<T>(some ? y * inv : 0.0f);
    }
    if (tid == 0 && a.lse) a.lse[blockIdx.x] = some ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <typename F>
cudaError_t with_dim(int dim, F &&f) {
    switch (dim) {
        case 32: return f(std::integral_constant<int, 32>{});
        case 64: return f(std::integral_constant<int, 64>{});
        case 96: return f(std::integral_constant<int, 96>{});
        case 128: return f(std::integral_constant<int, 128>{});
        default: return f(std::integral_constant<int, 256>{});
    }
}

cudaError_t launch_join(const JoinArgs &a, int dim, int dtype, cudaStream_t st) {
    const int64_t rows = (int64_t)a.B * a.tokens * a.heads;
    if (rows > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return with_dtype(dtype, [&](auto t) {
        return with_dim(dim, [&](auto d) {
            count_launches(1);
            return cudaLaunchKernelEx(&cfg, kv8_join_lists_kernel<decltype(t), decltype(d)::value>, a);
        });
    });
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Which kernel a call takes: up to this many query rows of a key/value head the one of few rows,
// which reads the cache at its rate by 16 rows of 16 bits (or 8 of f32) and again for as many more;
// beyond, 128 rows a tile.  Both in us, few rows then tiles, by 8 heads of 128 dims:
//                                 16 rows, bf16 (f16)     20 rows         |  f32 20 rows    32         48
//   16 sequences of 16384         132, 203 (131, 272)     233, 203 (272)  |  295, 445   299, 446   428, 446
//   16 of 2048                    36, 32 (36, 41)         61, 32 (41)     |  62, 59     65, 59     86, 60
//   one of 16384                  30, 24 (30, 28)         46, 24 (28)     |  46, 36     47, 37     55, 37
bool few(int64_t rows, int dtype) { return rows <= (dtype == BSG_F32 ? 32 : 16); }

// The workspace of one part of a call, largest over the types: a call takes the plan of its own.
constexpr int kDtypes[] = {BSG_F32, BSG_F16, BSG_BF16};
size_t part_floats(const bsg_kv8_cache &c, int64_t rows, int64_t B, int64_t positions, bool later) {
    size_t most = 0;
    for (const int dtype : kDtypes) {
        const KvPlan p = kv_plan(c, few(rows, dtype), dtype, rows, B, positions, positions, later);
        if (p.parts * (c.dim + 2) > most) most = p.parts * (c.dim + 2);
    }
    return most;
}

int64_t seen_positions(const bsg_kv8_cache &c, int64_t table_ld, int64_t tokens, int window, int sinks) {
    const int64_t all = table_ld * c.page_tokens, some = (int64_t)window + tokens + sinks + 3 * 128;
    return window && some < all ? some : all;
}

}  // namespace

size_t kv8_window_workspace_bytes(const bsg_kv8_cache &c, int64_t table_ld, int64_t B, int64_t T,
                                  int heads, int window, int sinks) {
    return up256(part_floats(c, T * (heads / c.heads), B, seen_positions(c, table_ld, T, window, sinks), false) * 4 + 1);
}

cudaError_t launch_kv8_attend_window(const bsg_kv8_cache &c, const int32_t *table, int64_t table_ld,
                                     const int32_t *lens, const int32_t *counts, const bsg_tokens &q,
                                     const bsg_tokens &out, int dtype, int64_t B, int64_t T,
                                     int heads, int window, int sinks, float scale, float *lse,
                                     void *ws, int32_t *dstatus, cudaStream_t st) {
    const int64_t rows = T * (heads / c.heads);
    const bool is_few = few(rows, dtype);
    // a CTA of tiles has 256 rows
    const int64_t share = heads / c.heads, some = 255 / share + 2;
    const KvPlan p = kv_plan(c, is_few, dtype, rows, B, seen_positions(c, table_ld, T, window, sinks),
                             seen_positions(c, table_ld, T < some ? T : some, window, sinks), false);
    KvCall a{c, table, table_ld, lens, counts, q, out, dtype, (int)T, heads, window, sinks, B, rows, scale, lse, 0,
             static_cast<float *>(ws), nullptr, dstatus};
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + p.parts * c.dim);
    cudaError_t e = is_few ? launch_few_window(a, p, st) : launch_tiles_window(a, p, st);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_join({out, c.heads, heads, (int)T, (int)B, nullptr, counts, 0, {a.part_o, nullptr},
                        {a.part_ml, nullptr}, {p.splits, 0}, lse},
                       c.dim, dtype, st);
}

size_t kv8_shared_workspace_bytes(const bsg_kv8_cache &c, int64_t prefix_pages, int64_t table_ld,
                                  int64_t B, int64_t T, int heads) {
    const int64_t rows = T * (heads / c.heads);
    return up256((part_floats(c, rows, B, table_ld * c.page_tokens, true) +
                  part_floats(c, B * rows, 1, prefix_pages * c.page_tokens, true)) * 4);
}

cudaError_t launch_kv8_attend_shared(const bsg_kv8_cache &c, const int32_t *prefix,
                                     int64_t prefix_pages, const int32_t *prefix_len,
                                     const int32_t *table, int64_t table_ld, const int32_t *lens,
                                     const bsg_tokens &q, const bsg_tokens &out, int dtype,
                                     int64_t B, int64_t T, int heads, float scale, float *lse,
                                     void *ws, int32_t *dstatus, cudaStream_t st) {
    const int64_t rows = T * (heads / c.heads);
    if (B * rows > INT32_MAX) return cudaErrorInvalidValue;
    const bool few_own = few(rows, dtype), few_pre = few(B * rows, dtype);
    const int64_t own_most = table_ld * c.page_tokens, pre_most = prefix_pages * c.page_tokens;
    const KvPlan own = kv_plan(c, few_own, dtype, rows, B, own_most, own_most, true);
    const KvPlan pre = kv_plan(c, few_pre, dtype, B * rows, 1, pre_most, pre_most, true);
    float *own_o = static_cast<float *>(ws), *pre_o = own_o + own.parts * c.dim;
    float2 *own_ml = reinterpret_cast<float2 *>(pre_o + pre.parts * c.dim), *pre_ml = own_ml + own.parts;
    KvCall a{c, table, table_ld, lens, nullptr, q, out, dtype, (int)T, heads, 0, 0, B, rows, scale, lse, 1,
             own_o, own_ml, dstatus};
    cudaError_t e = few_own ? launch_few_window(a, own, st) : launch_tiles_window(a, own, st);
    if (e != cudaSuccess) return e;
    a.table = prefix, a.table_ld = prefix_pages, a.lens = prefix_len, a.B = 1, a.rows = B * rows;
    a.part_o = pre_o, a.part_ml = pre_ml;
    e = few_pre ? launch_few_prefix(a, pre, st) : launch_tiles_prefix(a, pre, st);
    if (e != cudaSuccess) return e;
    return launch_join({out, c.heads, heads, (int)T, (int)B, lens, nullptr, table_ld * c.page_tokens, {own_o, pre_o},
                        {own_ml, pre_ml}, {own.splits, pre.splits}, lse},
                       c.dim, dtype, st);
}

}  // namespace bsg
