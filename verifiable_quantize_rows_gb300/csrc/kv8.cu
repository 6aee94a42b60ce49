// kv8.cu -- the int8 key/value cache: appending tokens, and attention over it.
//
// A page holds page_tokens tokens of every head; each page and head has one
// f32 scale for its keys and one for its values.  The codes follow the unit's
// ("Verification", section "The verified INT8 units", step 1: scale =
// max / 127 floored at 1e-8, floor(x inv + 0.5)) over a block of tokens in
// place of a row; the scale is one f32 product with f32(1/127).
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "bsg_internal.h"
#include "bsg_ptx.cuh"
#include "kv8_attend.cuh"
#include "serve.cuh"

namespace bsg {
namespace {

template <int N>
__device__ __forceinline__ float block_max(float x, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (N == 32) return x;
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < N / 32; ++i) x = fmaxf(x, red[i]);
    __syncthreads();
    return x;
}

template <int N>
__device__ __forceinline__ float block_sum(float x, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < N / 32; ++i) x += red[i];
    __syncthreads();
    return x;
}

// ---- append -----------------------------------------------------------------
//
// One CTA per touched page of a sequence, some of the heads, and side (keys or
// values); a warp where the new tokens are few.  A head's tokens are on their way
// while the one before it is stored.  A thread takes 8 values at a time and keeps kKept
// such pieces in registers between the maximum and the codes, so that new tokens
// are read once (up to 64 x 128 values a page; larger ones are read again, from
// L2), and sends for them before it knows where they go.
//
// Measured: prompts of 168 MB of bf16 keys and values 52 us (0.72 of the floor's rate; 58
// with a floor by comparison), 64 sequences' single tokens 3.6 us.  What bounds prompts:
// some 14 instructions a value (its share of the maximum, the conversion, the code and the
// packing) at 16 warps an SM, which issue in 0.64 of the cycles; single tokens: the launch and two dependent reads (the table,
// then the page's old scale).  (256 threads of 4 pieces: 55 to 61 us, the registers of 32
// warps spill; reading every token twice: 210.)

// 8 values as they are stored.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p, bool aligned) {
        if (aligned) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        } else {
            T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = p[i];
            memcpy(w, e, sizeof(w));
        }
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        T e[8];
        memcpy(e, w, sizeof(w));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
    }
    // Raises `top`, the largest |x| so far as bits (of 16-bit types, of the values
    // in each half): magnitudes are in order as whole numbers, Inf and NaN above all.
    __device__ __forceinline__ void raise(uint32_t &top) const {
        const uint32_t *b = reinterpret_cast<const uint32_t *>(w);
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i)
            top = sizeof(T) == 2 ? __vmaxu2(top, b[i] & 0x7fff7fffu) : max(top, b[i] & 0x7fffffffu);
    }
    static __device__ __forceinline__ float absmax(uint32_t top) {
        if (sizeof(T) == 4) return __uint_as_float(top);
        const unsigned short m = (unsigned short)max(top & 0xffffu, top >> 16);
        T e;
        memcpy(&e, &m, 2);
        return to_f32(e);
    }
};

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __byte_perm(unit_code(x[4 * i], inv), unit_code(x[4 * i + 1], inv), 0x0040);
        const uint32_t hi = __byte_perm(unit_code(x[4 * i + 2], inv), unit_code(x[4 * i + 3], inv), 0x0040);
        w[i] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint2(w[0], w[1]);
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 32 ? 1 : sizeof(T) == 2 ? 4 : 3)
    kv8_append_kernel(const __grid_constant__ bsg_kv8_cache c, const int32_t *__restrict__ table,
                      int64_t table_ld, const int32_t *__restrict__ starts,
                      const int32_t *__restrict__ counts, const __grid_constant__ bsg_tokens tk,
                      const __grid_constant__ bsg_tokens tv, int blocks, int tokens, int aligned,
                      int heads, int32_t *__restrict__ dstatus) {
    constexpr int kKept = kThreads == 32 ? 4 : 8;
    __shared__ float red[kThreads / 32];
    const int b = blockIdx.x / blocks, t = threadIdx.x;
    const int h0 = blockIdx.y * heads, h1 = min(c.heads, h0 + heads);
    const int start = starts[b], count = counts ? counts[b] : tokens;
    if (start < 0 || count < 0 || count > tokens) {
        if (t == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
        return;
    }
    const int P = c.page_tokens, D = c.dim, per = D / 8;  // pieces of a token
    const int64_t end = (int64_t)start + count;
    const int64_t j = start / P + blockIdx.x % blocks;  // the sequence's page
    if (j * P >= end) return;
    const int lo = (int)(start > j * P ? start - j * P : 0);  // new tokens: [lo, hi)
    const int hi = (int)(end < (j + 1) * P ? end - j * P : P);
    const bsg_tokens &tok = blockIdx.z ? tv : tk;
    const T *x = (const T *)tok.data + b * tok.stride_batch + (j * P - start) * tok.stride_token;
    const bool vec = aligned >> blockIdx.z & 1;
    // The thread's pieces: e0, e0 + kThreads ... (which is step_tokens tokens and
    // step_pieces pieces on).
    const int e0 = lo * per + t, e1 = hi * per;
    const int step_tokens = kThreads / per, step_pieces = kThreads % per;
    const int64_t step = step_tokens * tok.stride_token;
    auto each = [&](int h, int skip, auto &&f) {  // f(piece, its address), after the first `skip`
        int e = e0 + skip * kThreads, p = e % per;
        const T *at = x + h * tok.stride_head + (e / per) * tok.stride_token + p * 8;
        for (; e < e1; e += kThreads) {
            f(e, at);
            at += step + step_pieces * 8;
            if ((p += step_pieces) >= per) p -= per, at += tok.stride_token - per * 8;
        }
    };
    Raw8<T> kept[kKept], next[kKept];
    auto load = [&](int h) {
        int p = e0 % per;
        const T *at = x + h * tok.stride_head + (e0 / per) * tok.stride_token + p * 8;
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            if (e0 + i * kThreads < e1) next[i].load(at, vec);
            at += step + step_pieces * 8;
            if ((p += step_pieces) >= per) p -= per, at += tok.stride_token - per * 8;
        }
    };
    load(h0);

    int page = -1;
    if (j < table_ld) page = table[b * table_ld + j];
    if (page < 0 || page >= c.pages) {
        if (t == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
        return;
    }
    for (int h = h0; h < h1; ++h) {
#pragma unroll
        for (int i = 0; i < kKept; ++i) kept[i] = next[i];
        if (h + 1 < h1) load(h + 1);
        const int64_t ph = (int64_t)page * c.heads + h;
        uint2 *codes = reinterpret_cast<uint2 *>((blockIdx.z ? c.v : c.k) + ph * P * D);
        float *scale = (blockIdx.z ? c.v_scale : c.k_scale) + ph;
        const float old = lo > 0 ? *scale : 0.0f;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kKept; ++i)
            if (e0 + i * kThreads < e1) kept[i].raise(top);
        each(h, kKept, [&](int, const T *at) {
            Raw8<T> raw;
            raw.load(at, vec);
            raw.raise(top);
        });
        const float most = Raw8<T>::absmax(top);
        if (!(most < INFINITY)) set_status(dstatus, BSG_DSTATUS_NONFINITE);
        float s = kv8_scale(block_max<kThreads>(most, red));
        __syncwarp();  // all have read the old scale
        if (old < s) {
            if (lo > 0) {
                const float r = __fdiv_rn(old, s);
                for (int e = t; e < lo * per; e += kThreads) {
                    const uint2 w = codes[e];
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)((k < 4 ? w.x : w.y) >> (k % 4 * 8));
                    codes[e] = codes8(v, r);
                }
            }
            if (t == 0) *scale = s;
        } else {
            s = old;
        }
        const float inv = __fdiv_rn(1.0f, s);
        auto store = [&](const Raw8<T> &raw, int e) {
            float v[8];
            raw.values(v);
            codes[e] = codes8(v, inv);
        };
#pragma unroll
        for (int i = 0; i < kKept; ++i)
            if (e0 + i * kThreads < e1) store(kept[i], e0 + i * kThreads);
        each(h, kKept, [&](int e, const T *at) {
            Raw8<T> raw;
            raw.load(at, vec);
            store(raw, e);
        });
    }
}

// ---- attention: kv8_attend.cuh; the join of its chunks ------------------------------

// Joins the chunks of one row: grid (rows, heads, B), a column of four and
// every kSides-th chunk to a thread.
constexpr int kJoin = 128;
template <int D>
__global__ void __launch_bounds__(kJoin) kv8_join_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int kCols = D / 4, kSides = kJoin / kCols;
    __shared__ float f_s[kMaxSplits], red[kJoin / 32];
    __shared__ float4 o_s[kSides][kCols];
    const int r = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int all = (length_of(a, b, false) + 15) / 16;
    int n = 0;  // chunks that begin within the length
    for (int i0 = 0; i0 < a.splits; i0 += kJoin)
        n += __syncthreads_count(i0 + tid < a.splits && chunk_begin(a, i0 + tid) < all);
    griddep_wait();  // every block, so that this grid never ends before the one it joins
    if (all <= chunk_begin(a, 1)) return;  // finished where it was computed
    const int64_t part = (((int64_t)b * a.c.heads + hk) * a.rows + r) * a.splits;
    const float2 *ml = a.part_ml + part;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + part * D);
    const int col = tid % kCols, side = tid / kCols;
    // the first outputs are on their way while the weights are found
    constexpr int kAhead = 4;
    float4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (side < kSides && side + i * kSides < n) v[i] = po[(int64_t)(side + i * kSides) * kCols + col];
    float m = kRefNone;
    for (int i = tid; i < n; i += kJoin) m = fmaxf(m, ml[i].x);
    m = block_max<kJoin>(m, red);
    float l = 0.0f;
    for (int i = tid; i < n; i += kJoin) {
        const float2 x = ml[i];
        f_s[i] = exp2_fast(x.x - m);
        l = fmaf(x.y, f_s[i], l);
    }
    l = block_sum<kJoin>(l, red);  // and f_s is complete
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = side; i0 < n && side < kSides; i0 += kAhead * kSides) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int at = i0 + i * kSides, then = at + kAhead * kSides;
            if (at >= n) break;
            const float f = f_s[at];
            o.x = fmaf(v[i].x, f, o.x), o.y = fmaf(v[i].y, f, o.y);
            o.z = fmaf(v[i].z, f, o.z), o.w = fmaf(v[i].w, f, o.w);
            if (then < n) v[i] = po[(int64_t)then * kCols + col];
        }
    }
    if (side < kSides) o_s[side][col] = o;
    __syncthreads();
    for (int d = tid; d < D; d += kJoin) {
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < kSides; ++i) y += reinterpret_cast<const float *>(&o_s[i][d / 4])[d % 4];
        store_row(a, b, hk, r, d, y, m, l);
    }
}

}  // namespace

cudaError_t launch_kv8_append(const bsg_kv8_cache &c, const int32_t *table, int64_t table_ld,
                              const int32_t *starts, const int32_t *counts, const bsg_tokens &k,
                              const bsg_tokens &v, int dtype, int64_t B, int64_t T,
                              int32_t *dstatus, cudaStream_t st) {
    // T tokens from any position touch at most this many pages
    const int64_t blocks = (T - 2 + c.page_tokens) / c.page_tokens + 1;
    if (B * blocks > INT32_MAX) return cudaErrorInvalidValue;
    return with_dtype(dtype, [&](auto t) {
        using E = decltype(t);
        auto on16 = [](const bsg_tokens &x) {
            return (reinterpret_cast<uintptr_t>(x.data) | (uintptr_t)(x.stride_batch * (int64_t)sizeof(E)) |
                    (uintptr_t)(x.stride_token * (int64_t)sizeof(E)) |
                    (uintptr_t)(x.stride_head * (int64_t)sizeof(E))) % 16 == 0;
        };
        const int aligned = (int)on16(k) | (int)on16(v) << 1;
        // few tokens: a warp to a head; prompts: as many heads as leave four CTAs for
        // each of four places on an SM
        const bool few = T * c.dim <= 1024;
        int64_t heads = few ? 1 : 2 * B * blocks * c.heads / (16 * (int64_t)device_sm_count());
        heads = heads < 1 ? 1 : heads > c.heads ? c.heads : heads;
        const int64_t groups = (c.heads + heads - 1) / heads;
        heads = (c.heads + groups - 1) / groups;  // alike
        const dim3 grid((unsigned)(B * blocks), (unsigned)groups, 2);
        if (few)
            kv8_append_kernel<E, 32><<<grid, 32, 0, st>>>(c, table, table_ld, starts, counts, k, v, (int)blocks,
                                                          (int)T, aligned, 1, dstatus);
        else
            kv8_append_kernel<E, 128><<<grid, 128, 0, st>>>(c, table, table_ld, starts, counts, k, v, (int)blocks,
                                                            (int)T, aligned, (int)heads, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

size_t kv8_attend_workspace_bytes(const bsg_kv8_cache &c, int64_t table_ld, int64_t B, int64_t T,
                                  int heads) {
    size_t most = 256;
    for (int parts = 1; parts <= 2; ++parts) {
        const AttendPlan p = attend_plan(c, table_ld, B, T, heads, parts);
        const size_t n = (size_t)B * c.heads * p.rows * p.splits * (c.dim * 4 + 8);
        if (p.splits > 1 && n > most) most = n;
    }
    return (most + 255) / 256 * 256;
}

// The join, launched while the attention still runs: its blocks wait for it.
template <int D>
static cudaError_t launch_join(const AttendArgs &a, const AttendPlan &p, int64_t B, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows, (unsigned)a.c.heads, (unsigned)B);
    cfg.blockDim = dim3(kJoin);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kv8_join_kernel<D>, a);
}

template <int D>
static cudaError_t launch_attend_dim(const AttendArgs &a, const AttendPlan &p, int64_t B, cudaStream_t st) {
    const cudaError_t e = launch_attend_nt<D, kWhole>(a, p, B, st);
    return e == cudaSuccess && p.splits > 1 ? launch_join<D>(a, p, B, st) : e;
}

cudaError_t launch_kv8_attend(const bsg_kv8_cache &c, const int32_t *table, int64_t table_ld,
                              const int32_t *lens, const bsg_tokens &q, const bsg_tokens &out,
                              int dtype, int64_t B, int64_t T, int heads, float scale, float *lse,
                              void *ws, int32_t *dstatus, cudaStream_t st) {
    const AttendPlan p = attend_plan(c, table_ld, B, T, heads, dtype == BSG_F32 ? 2 : 1);
    AttendArgs a{c, table, table_ld, lens, q, out, dtype, (int)T, heads, p.rows, p.row_tiles,
                 p.width, p.splits, scale, lse, nullptr, nullptr, dstatus, nullptr, 0, 0, 0};
    a.part_o = static_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)B * c.heads * p.rows * p.splits * c.dim);
    switch (c.dim) {
        case 32: return launch_attend_dim<32>(a, p, B, st);
        case 64: return launch_attend_dim<64>(a, p, B, st);
        case 96: return launch_attend_dim<96>(a, p, B, st);
        case 128: return launch_attend_dim<128>(a, p, B, st);
        default: return launch_attend_dim<256>(a, p, B, st);
    }
}

}  // namespace bsg
