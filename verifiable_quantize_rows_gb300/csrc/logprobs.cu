// logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of logits, and their gradient.
//
//   lse = m + log S,  S = sum_j e_j,  e_j = exp(x_j - m),  m = max_j x_j;
//   entropy = log S - (sum_j e_j (x_j - m)) / S;
//   dx_j = g_lp ([j = t] - p_j) - g_H p_j (x_j - lse + H).
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "serve.cuh"

namespace bsg {
namespace {

// One CTA per row; one read for the maximum, one for the sums, and one for
// each of the top alternatives.
template <typename T>
__global__ void __launch_bounds__(256)
    logprobs_kernel(const T *__restrict__ logits, int64_t V, int64_t ldl,
                    const int64_t *__restrict__ target, int top, float *__restrict__ logprob,
                    float *__restrict__ entropy, float *__restrict__ lse,
                    float *__restrict__ top_logprob, int32_t *__restrict__ top_id,
                    int32_t *__restrict__ dstatus) {
    __shared__ float red[8], red2[8];
    __shared__ int redi[8];
    const int64_t row = blockIdx.x;
    const T *x = logits + row * ldl;
    const int t = threadIdx.x, w = t / 32;
    auto best = [&](float v, int i) {  // the largest value, then the lowest index
        for (int o = 16; o; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, v, o);
            const int oi = __shfl_xor_sync(0xffffffffu, i, o);
            if (ov > v || (ov == v && oi < i)) v = ov, i = oi;
        }
        __syncthreads();
        if (t % 32 == 0) red[w] = v, redi[w] = i;
        __syncthreads();
        v = red[0], i = redi[0];
        for (int k = 1; k < 8; ++k)
            if (red[k] > v || (red[k] == v && redi[k] < i)) v = red[k], i = redi[k];
        return make_float2(v, __int_as_float(i));
    };
    float m = -INFINITY;
    bool bad = false;
    for (int64_t j = t; j < V; j += 256) {
        const float v = to_f32(x[j]);
        bad |= !(v < INFINITY);
        m = fmaxf(m, v);
    }
    if (bad) set_status(dstatus, BSG_DSTATUS_NONFINITE);
    m = best(m, 0).x;
    float s = 0.0f, a = 0.0f;
    for (int64_t j = t; j < V; j += 256) {
        const float d = to_f32(x[j]) - m, e = expf(d);
        s += e;
        if (e > 0.0f) a = fmaf(e, d, a);
    }
    for (int o = 16; o; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        a += __shfl_xor_sync(0xffffffffu, a, o);
    }
    __syncthreads();
    if (t % 32 == 0) red[w] = s, red2[w] = a;
    __syncthreads();
    s = a = 0.0f;
    for (int k = 0; k < 8; ++k) s += red[k], a += red2[k];
    const bool none = m == -INFINITY;  // every logit is -inf
    const float logs = none ? 0.0f : logf(s);
    if (t == 0) {
        if (lse) lse[row] = m + logs;
        if (entropy) entropy[row] = none ? 0.0f : logs - a / s;
        if (logprob) {
            const int64_t g = target ? target[row] : -1;
            if (g >= V) set_status(dstatus, BSG_DSTATUS_RANGE);
            logprob[row] = g < 0 ? 0.0f
                                 : g >= V ? NAN : none ? -INFINITY : to_f32(x[g]) - m - logs;
        }
    }
    float lv = INFINITY;
    int li = -1;
    for (int k = 0; k < top; ++k) {
        float v = -INFINITY;
        int i = INT32_MAX;
        for (int64_t j = t; j < V; j += 256) {
            const float y = to_f32(x[j]);
            if (y < lv || (y == lv && j > li))
                if (y > v || i == INT32_MAX) v = y, i = (int)j;
        }
        const float2 r = best(v, i);
        lv = r.x;
        li = __float_as_int(r.y);
        if (t == 0) {
            top_logprob[row * top + k] = none ? -INFINITY : lv - m - logs;
            top_id[row * top + k] = li;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
    logprobs_backward_kernel(const T *logits, int64_t V, int64_t ldl,
                             const int64_t *__restrict__ target, const float *__restrict__ lse,
                             const float *__restrict__ entropy,
                             const float *__restrict__ g_logprob,
                             const float *__restrict__ g_entropy, T *dlogits, int64_t ldd,
                             int32_t *__restrict__ dstatus) {
    const int64_t row = blockIdx.x;
    const T *x = logits + row * ldl;
    T *dx = dlogits + row * ldd;
    const int64_t g = target ? target[row] : -1;
    const float L = lse[row], H = g_entropy ? entropy[row] : 0.0f;
    const float gl = g_logprob && g >= 0 ? g_logprob[row] : 0.0f;
    const float gh = g_entropy ? g_entropy[row] : 0.0f;
    if (g >= V && threadIdx.x == 0) set_status(dstatus, BSG_DSTATUS_RANGE);
    bool bad = false;
    for (int64_t j = threadIdx.x; j < V; j += 256) {
        const float v = to_f32(x[j]), lp = v - L, p = expf(lp);
        bad |= !(v < INFINITY);
        float d = p > 0.0f ? -p * fmaf(gh, lp + H, gl) : 0.0f;
        if (j == g) d += gl;
        if (L == -INFINITY) d = 0.0f;
        if (g >= V) d = NAN;
        dx[j] = from_f32<T>(d);
    }
    if (bad) set_status(dstatus, BSG_DSTATUS_NONFINITE);
}

}  // namespace

cudaError_t launch_logprobs(const void *logits, int dtype, int64_t M, int64_t V, int64_t ldl,
                            const int64_t *target, int top, float *logprob, float *entropy,
                            float *lse, float *top_logprob, int32_t *top_id, int32_t *dstatus,
                            cudaStream_t st) {
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        logprobs_kernel<T><<<(unsigned)M, 256, 0, st>>>((const T *)logits, V, ldl, target, top,
                                                        logprob, entropy, lse, top_logprob, top_id,
                                                        dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

cudaError_t launch_logprobs_backward(const void *logits, int dtype, int64_t M, int64_t V,
                                     int64_t ldl, const int64_t *target, const float *lse,
                                     const float *entropy, const float *g_logprob,
                                     const float *g_entropy, void *dlogits, int64_t ldd,
                                     int32_t *dstatus, cudaStream_t st) {
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        logprobs_backward_kernel<T><<<(unsigned)M, 256, 0, st>>>(
            (const T *)logits, V, ldl, target, lse, entropy, g_logprob, g_entropy, (T *)dlogits,
            ldd, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace bsg
