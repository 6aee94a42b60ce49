// kv8.cu -- the int8 key/value cache: appending tokens, and attention over it.
//
// A page holds page_tokens tokens of every head; each page and head has one
// f32 scale for its keys and one for its values.  The codes follow the unit's
// ("Verification", section "The verified INT8 units", step 1: scale =
// max / 127 floored at 1e-8, floor(x inv + 0.5)) over a block of tokens in
// place of a row; the scale is one f32 product with f32(1/127).
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "serve.cuh"

namespace bsg {
namespace {

template <int N>
__device__ __forceinline__ float block_max(float x, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
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

// One CTA per touched page of a sequence, head, and side (keys or values).
template <typename T>
__global__ void __launch_bounds__(128)
    kv8_append_kernel(bsg_kv8_cache c, const int32_t *__restrict__ table, int64_t table_ld,
                      const int32_t *__restrict__ starts, const int32_t *__restrict__ counts,
                      bsg_tokens tk, bsg_tokens tv, int blocks, int tokens,
                      int32_t *__restrict__ dstatus) {
    __shared__ float red[4];
    const int b = blockIdx.x / blocks, h = blockIdx.y, t = threadIdx.x;
    const int start = starts[b], count = counts ? counts[b] : tokens;
    if (start < 0 || count < 0 || count > tokens) {
        if (t == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
        return;
    }
    const int P = c.page_tokens, D = c.dim;
    const int64_t end = (int64_t)start + count;
    const int64_t j = start / P + blockIdx.x % blocks;  // the sequence's page
    if (j * P >= end) return;
    int page = -1;
    if (j < table_ld) page = table[b * table_ld + j];
    if (page < 0 || page >= c.pages) {
        if (t == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
        return;
    }
    const bsg_tokens &tok = blockIdx.z ? tv : tk;
    const int64_t ph = (int64_t)page * c.heads + h;
    int8_t *codes = (blockIdx.z ? c.v : c.k) + ph * P * D;
    float *scale = (blockIdx.z ? c.v_scale : c.k_scale) + ph;
    const int lo = (int)(start > j * P ? start - j * P : 0);              // new tokens: [lo, hi)
    const int hi = (int)(end < (j + 1) * P ? end - j * P : P);
    const T *x = (const T *)tok.data + b * tok.stride_batch + h * tok.stride_head +
                 (j * P - start) * tok.stride_token;
    float m = 0.0f;
    bool bad = false;
    for (int i = lo * D + t; i < hi * D; i += 128) {
        const float v = to_f32(x[(i / D) * tok.stride_token + i % D]);
        bad |= !isfinite(v);
        m = fmaxf(m, fabsf(v));
    }
    if (bad) set_status(dstatus, BSG_DSTATUS_NONFINITE);
    m = block_max<128>(m, red);
    float s = kv8_scale(m);
    if (lo > 0) {
        const float old = *scale;
        if (old < s) {
            const float r = __fdiv_rn(old, s);
            for (int i = t; i < lo * D; i += 128) codes[i] = (int8_t)unit_code(codes[i], r);
        } else {
            s = old;
        }
    }
    const float inv = __fdiv_rn(1.0f, s);
    for (int i = lo * D + t; i < hi * D; i += 128)
        codes[i] = (int8_t)unit_code(to_f32(x[(i / D) * tok.stride_token + i % D]), inv);
    __syncthreads();  // every thread has read the old scale
    if (t == 0) *scale = s;
}

// One CTA per query row: chunks of 128 positions with a running maximum.
template <typename T>
__global__ void __launch_bounds__(128)
    kv8_attend_kernel(bsg_kv8_cache c, const int32_t *__restrict__ table, int64_t table_ld,
                      const int32_t *__restrict__ lens, bsg_tokens q, bsg_tokens out, int tokens,
                      int heads, float scale, float *__restrict__ lse,
                      int32_t *__restrict__ dstatus) {
    __shared__ float red[4], p_s[128], q_s[256];
    __shared__ int page_s[128];
    const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
    const int P = c.page_tokens, D = c.dim, hk = h / (heads / c.heads);
    int len = lens[b];
    if (len < 0 || len > table_ld * P) {
        if (t == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
        len = len < 0 ? 0 : (int)(table_ld * P);
    }
    const int see = len - tokens + i + 1;
    const T *qr = (const T *)q.data + b * q.stride_batch + i * q.stride_token + h * q.stride_head;
    bool bad = false;
    for (int d = t; d < D; d += 128) {
        q_s[d] = to_f32(qr[d]);
        bad |= !isfinite(q_s[d]);
    }
    if (bad) set_status(dstatus, BSG_DSTATUS_NONFINITE);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
    for (int j0 = 0; j0 < see; j0 += 128) {
        const int j = j0 + t;
        float s = -INFINITY;
        int page = -1;
        if (j < see) {
            page = table[b * table_ld + j / P];
            if (page < 0 || page >= c.pages) {
                set_status(dstatus, BSG_DSTATUS_RANGE);
                page = -1;
            } else {
                const int64_t ph = (int64_t)page * c.heads + hk;
                const int8_t *k = c.k + (ph * P + j % P) * D;
                float a = 0.0f;
                for (int d = 0; d < D; ++d) a = fmaf(q_s[d], (float)k[d], a);
                s = a * c.k_scale[ph] * scale;
            }
        }
        const float top = fmaxf(m, block_max<128>(s, red));
        const float p = top == -INFINITY ? 0.0f : expf(s - top);
        const float keep = m == -INFINITY ? 0.0f : expf(m - top);
        m = top;
        l = l * keep + block_sum<128>(p, red);
        p_s[t] = p;
        page_s[t] = page;
        __syncthreads();
        const int n = min(128, see - j0);
        for (int u = 0; u < 2; ++u) {
            const int d = t + 128 * u;
            if (d >= D) break;
            o[u] *= keep;
            for (int e = 0; e < n; ++e) {
                if (page_s[e] < 0) continue;
                const int64_t ph = (int64_t)page_s[e] * c.heads + hk;
                o[u] = fmaf(p_s[e] * c.v_scale[ph], (float)c.v[(ph * P + (j0 + e) % P) * D + d],
                            o[u]);
            }
        }
        __syncthreads();
    }
    T *orow = (T *)out.data + b * out.stride_batch + i * out.stride_token + h * out.stride_head;
    for (int u = 0; u < 2; ++u)
        if (t + 128 * u < D) orow[t + 128 * u] = from_f32<T>(l > 0.0f ? o[u] / l : 0.0f);
    if (lse && t == 0)
        lse[((int64_t)b * tokens + i) * heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
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
        const dim3 grid((unsigned)(B * blocks), (unsigned)c.heads, 2);
        kv8_append_kernel<E><<<grid, 128, 0, st>>>(c, table, table_ld, starts, counts, k, v,
                                                   (int)blocks, (int)T, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

size_t kv8_attend_workspace_bytes(const bsg_kv8_cache &, int64_t, int64_t, int64_t, int) {
    return 256;
}

cudaError_t launch_kv8_attend(const bsg_kv8_cache &c, const int32_t *table, int64_t table_ld,
                              const int32_t *lens, const bsg_tokens &q, const bsg_tokens &out,
                              int dtype, int64_t B, int64_t T, int heads, float scale, float *lse,
                              void *, int32_t *dstatus, cudaStream_t st) {
    return with_dtype(dtype, [&](auto t) {
        using E = decltype(t);
        const dim3 grid((unsigned)heads, (unsigned)T, (unsigned)B);
        kv8_attend_kernel<E><<<grid, 128, 0, st>>>(c, table, table_ld, lens, q, out, (int)T, heads,
                                                   scale, lse, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace bsg
