// wcols.cu -- products of any number of tokens with a weight stored as int8 codes and
// one scale per column: each token quantized by itself, exact sums of code products.
//
// "The verified INT8 units", steps 1 to 3, on a weight that keeps its codes: step 1 for
// the tokens alone, into the f16 operand that the tensor-core GEMM reads (every code is
// exact in f16), the weight's codes laid out as the other operand, then the GEMM.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "serve.cuh"

namespace bsg {
namespace {

constexpr int kTokenThreads = 256;

// Step 1 of one token, a CTA each.
template <typename T>
__global__ void __launch_bounds__(kTokenThreads)
    wcols_tokens_kernel(const T *__restrict__ X, int64_t ldx, int K, int ldk, __half *__restrict__ op,
                        float *__restrict__ scale, unsigned int *ticket, int32_t *dstatus) {
    __shared__ uint32_t red[kTokenThreads / 32];
    const int64_t row = blockIdx.x;
    const T *x = X + row * ldx;
    uint32_t m = 0;  // the largest |x|, as bits: Inf and NaN are the largest of all
    for (int k = threadIdx.x; k < K; k += kTokenThreads)
        m = max(m, __float_as_uint(to_f32(x[k])) & 0x7fffffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTokenThreads / 32; ++i) m = max(m, red[i]);
    // the unit's quotients, whose f32 divisions equal the f64 ones rounded
    const float s = fmaxf(__fdiv_rn(__uint_as_float(m), 127.0f), 1e-8f), inv = __fdiv_rn(1.0f, s);
    for (int k = threadIdx.x; k < ldk; k += kTokenThreads)
        op[row * ldk + k] = __int2half_rn(k < K ? (int)(int8_t)unit_code(to_f32(x[k]), inv) : 0);
    if (threadIdx.x == 0) {
        scale[row] = s;
        if (m >= 0x7f800000u) set_status(dstatus, BSG_DSTATUS_NONFINITE);
        if (row == 0) ticket[0] = ticket[1] = 0;
    }
}

struct Layout {
    int64_t ldk;
    size_t tokens, weights, token_scale, col_scale, ticket, bytes;
};
Layout layout(int64_t M, int64_t N, int64_t K) {
    Layout l;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.ldk = operand_ld(K);
    l.tokens = 0;
    l.weights = up((size_t)M * l.ldk * 2);
    l.token_scale = l.weights + up((size_t)N * l.ldk * 2);
    l.col_scale = l.token_scale + up((size_t)round_up(M, kBM) * 4);
    l.ticket = l.col_scale + up((size_t)(round_up(N, kBN) + kBN) * 4);
    l.bytes = l.ticket + 256;
    return l;
}

}  // namespace

size_t wcols_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) { return layout(M, N, K).bytes; }

cudaError_t launch_wcols_matmul(const void *X, int dtype, int64_t ldx, const int8_t *Q, int64_t ldq,
                                const float *scale, int64_t M, int64_t N, int64_t K, int relu,
                                void *Y, int64_t ldy, void *ws, int32_t *dstatus, cudaStream_t st) {
    const Layout l = layout(M, N, K);
    uint8_t *w = static_cast<uint8_t *>(ws);
    __half *aop = reinterpret_cast<__half *>(w + l.tokens), *bop = reinterpret_cast<__half *>(w + l.weights);
    float *sa = reinterpret_cast<float *>(w + l.token_scale), *sb = reinterpret_cast<float *>(w + l.col_scale);
    unsigned int *ticket = reinterpret_cast<unsigned int *>(w + l.ticket);
    cudaError_t e = with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        wcols_tokens_kernel<T><<<(unsigned)M, kTokenThreads, 0, st>>>(static_cast<const T *>(X), ldx, (int)K,
                                                                      (int)l.ldk, aop, sa, ticket, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    // the GEMM reads whole tiles of scales
    e = cudaMemcpyAsync(sb, scale, (size_t)N * 4, cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return e;
    e = launch_i8_cols_to_half(Q, K, N, ldq, bop, l.ldk, st);
    if (e != cudaSuccess) return e;
    return launch_gemm_tc(aop, bop, M, N, K, sa, sb, relu, dtype == BSG_F32 ? 0 : dtype == BSG_F16 ? 2 : 3, Y,
                          ldy, dstatus, ticket, st);
}

}  // namespace bsg
