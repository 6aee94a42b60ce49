// kv8_more.cu -- attention over the int8 cache for any number of query tokens through a
// window with sinks, and behind a prefix that all sequences share.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "serve.cuh"

namespace bsg {
namespace {

struct Args {
    bsg_kv8_cache c;
    const int32_t *table, *lens, *counts, *prefix, *prefix_len;
    int64_t table_ld, prefix_pages;
    bsg_tokens q, out;
    int tokens, heads, window, sinks;
    float scale;
    float *lse;
    int32_t *dstatus;
};

// A warp to a query row, a running maximum and sum.
template <typename T, int D>
__global__ void __launch_bounds__(128) rows_kernel(const __grid_constant__ Args a, int64_t rows) {
    const int lane = threadIdx.x % 32, P = a.c.page_tokens;
    const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (row >= rows) return;
    const int h = (int)(row % a.heads), t = (int)(row / a.heads % a.tokens);
    const int64_t b = row / a.heads / a.tokens;
    const int hk = h / (a.heads / a.c.heads);
    const int count = a.counts ? a.counts[b] : a.tokens;
    if (count < 0 || count > a.tokens) {
        if (lane == 0) set_status(a.dstatus, BSG_DSTATUS_RANGE);
        return;
    }
    if (t >= count) return;
    const int64_t most = a.table_ld * P;
    int64_t len = a.lens[b];
    if (len < 0 || len > most) {
        if (lane == 0) set_status(a.dstatus, BSG_DSTATUS_RANGE);
        len = len < 0 ? 0 : most;
    }
    const int64_t pos = len - count + t;
    float q[D / 32], o[D / 32];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        q[i] = to_f32(static_cast<const T *>(a.q.data)[b * a.q.stride_batch + t * a.q.stride_token +
                                                       h * a.q.stride_head + lane + 32 * i]);
        bad |= !isfinite(q[i]);
        o[i] = 0.0f;
    }
    if (bad) set_status(a.dstatus, BSG_DSTATUS_NONFINITE);
    float m = -INFINITY, l = 0.0f;
    auto see = [&](const int32_t *table, int64_t from, int64_t to) {
        for (int64_t j = from; j < to; ++j) {
            const int page = table[j / P];
            if (page < 0 || page >= a.c.pages) {
                if (lane == 0) set_status(a.dstatus, BSG_DSTATUS_RANGE);
                continue;
            }
            const int64_t ph = (int64_t)page * a.c.heads + hk, at = (ph * P + j % P) * D + lane;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) s = fmaf(q[i], (float)a.c.k[at + 32 * i], s);
#pragma unroll
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= a.scale * a.c.k_scale[ph];
            const float n = fmaxf(m, s), keep = expf(m - n), p = expf(s - n), vs = a.c.v_scale[ph];
            m = n;
            l = fmaf(l, keep, p);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], keep, p * vs * (float)a.c.v[at + 32 * i]);
        }
    };
    if (pos >= 0) {
        if (a.prefix) {
            int64_t n = *a.prefix_len;
            if (n < 0 || n > a.prefix_pages * P) {
                if (lane == 0) set_status(a.dstatus, BSG_DSTATUS_RANGE);
                n = n < 0 ? 0 : a.prefix_pages * P;
            }
            see(a.prefix, 0, n);
        }
        const int64_t low = a.window && pos >= a.window ? pos - a.window + 1 : 0;
        see(a.table + b * a.table_ld, 0, low < a.sinks ? low : a.sinks);
        see(a.table + b * a.table_ld, low, pos + 1);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        static_cast<T *>(a.out.data)[b * a.out.stride_batch + t * a.out.stride_token + h * a.out.stride_head +
                                     lane + 32 * i] = from_f32<T>(l > 0.0f || l != l ? o[i] / l : 0.0f);
    if (lane == 0 && a.lse)
        a.lse[row] = l > 0.0f || l != l ? m + logf(l) : -INFINITY;
}

cudaError_t launch(const Args &a, int dtype, int64_t B, cudaStream_t st) {
    const int64_t rows = B * a.tokens * a.heads;
    if ((rows + 3) / 4 > INT32_MAX) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        switch (a.c.dim) {
            case 32: rows_kernel<T, 32><<<grid, 128, 0, st>>>(a, rows); break;
            case 64: rows_kernel<T, 64><<<grid, 128, 0, st>>>(a, rows); break;
            case 96: rows_kernel<T, 96><<<grid, 128, 0, st>>>(a, rows); break;
            case 128: rows_kernel<T, 128><<<grid, 128, 0, st>>>(a, rows); break;
            default: rows_kernel<T, 256><<<grid, 128, 0, st>>>(a, rows);
        }
        count_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace

size_t kv8_window_workspace_bytes(const bsg_kv8_cache &, int64_t, int64_t, int64_t, int, int, int) {
    return 256;
}

cudaError_t launch_kv8_attend_window(const bsg_kv8_cache &c, const int32_t *table, int64_t table_ld,
                                     const int32_t *lens, const int32_t *counts, const bsg_tokens &q,
                                     const bsg_tokens &out, int dtype, int64_t B, int64_t T,
                                     int heads, int window, int sinks, float scale, float *lse,
                                     void *ws, int32_t *dstatus, cudaStream_t st) {
    return launch({c, table, lens, counts, nullptr, nullptr, table_ld, 0, q, out, (int)T, heads, window,
                   sinks, scale, lse, dstatus},
                  dtype, B, st);
}

size_t kv8_shared_workspace_bytes(const bsg_kv8_cache &, int64_t, int64_t, int64_t, int64_t, int) {
    return 256;
}

cudaError_t launch_kv8_attend_shared(const bsg_kv8_cache &c, const int32_t *prefix,
                                     int64_t prefix_pages, const int32_t *prefix_len,
                                     const int32_t *table, int64_t table_ld, const int32_t *lens,
                                     const bsg_tokens &q, const bsg_tokens &out, int dtype,
                                     int64_t B, int64_t T, int heads, float scale, float *lse,
                                     void *ws, int32_t *dstatus, cudaStream_t st) {
    return launch({c, table, lens, nullptr, prefix, prefix_len, table_ld, prefix_pages, q, out, (int)T,
                   heads, 0, 0, scale, lse, dstatus},
                  dtype, B, st);
}

}  // namespace bsg
