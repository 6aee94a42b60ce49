// wgroups.cu -- int4 weights with one scale per group of rows and column: the
// storage, and products of a few rows with it.
//
// The storage is wquant.cu's scheme ("Precision" manual, section "Integer
// weights") on blocks of `group` rows: s = absmax / 7 rounded to f32, codes
// the integer nearest w / s, ties to even, all-zero blocks s = 0.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsg_internal.h"
#include "serve.cuh"
#include "wq_round.cuh"

namespace bsg {
namespace {

// One thread per byte column (two weight columns) of one group: the maxima of
// its rows, then the codes from a second read (L2).
__global__ void __launch_bounds__(128)
    wquant_groups_kernel(const float *__restrict__ W, int64_t K, int64_t N, int64_t ldw,
                         int64_t group, uint8_t *__restrict__ Q, int64_t ldq,
                         float *__restrict__ scale, int64_t lds, int32_t *__restrict__ dstatus) {
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (2 * c >= N) return;
    const bool two = 2 * c + 1 < N;
    const int64_t groups = (K + group - 1) / group;
    for (int64_t g = blockIdx.y; g < groups; g += gridDim.y) {
        const int64_t k0 = g * group, k1 = k0 + group < K ? k0 + group : K;
        uint32_t m0 = 0, m1 = 0;
        for (int64_t k = k0; k < k1; ++k) {
            const float *row = W + k * ldw + 2 * c;
            m0 = max(m0, __float_as_uint(row[0]) & 0x7fffffffu);
            if (two) m1 = max(m1, __float_as_uint(row[1]) & 0x7fffffffu);
        }
        if (m0 >= 0x7f800000u || m1 >= 0x7f800000u) set_status(dstatus, BSG_DSTATUS_NONFINITE);
        const float s0 = __fdiv_rn(__uint_as_float(m0), 7.0f);
        const float s1 = __fdiv_rn(__uint_as_float(m1), 7.0f);
        scale[g * lds + 2 * c] = s0;
        if (two) scale[g * lds + 2 * c + 1] = s1;
        const bool u0 = s0 != 0.0f && isfinite(s0), u1 = s1 != 0.0f && isfinite(s1);
        const float r0 = u0 ? __frcp_rn(s0) : 0.0f, r1 = u1 ? __frcp_rn(s1) : 0.0f;
        for (int64_t k = k0; k < k1; ++k) {
            const float *row = W + k * ldw + 2 * c;
            const int q0 = u0 ? wq_round_quotient(row[0], s0, r0, 7) : 0;
            const int q1 = u1 && two ? wq_round_quotient(row[1], s1, r1, 7) : 0;
            Q[k * ldq + c] = (uint8_t)((q0 & 15) | ((q1 & 15) << 4));
        }
    }
}

// One thread per byte column and row of X: the plain sum over k.
template <typename T>
__global__ void __launch_bounds__(128)
    wgroups_matvec_kernel(const T *__restrict__ X, int64_t ldx, const uint8_t *__restrict__ Q,
                          int64_t ldq, const float *__restrict__ scale, int64_t lds,
                          int64_t group, int64_t N, int64_t K, int relu, T *__restrict__ Y,
                          int64_t ldy, int32_t *__restrict__ dstatus) {
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (2 * c >= N) return;
    const T *x = X + blockIdx.y * ldx;
    const bool two = 2 * c + 1 < N;
    float y0 = 0.0f, y1 = 0.0f;
    bool bad = false;
    for (int64_t k0 = 0, g = 0; k0 < K; k0 += group, ++g) {
        const int64_t k1 = k0 + group < K ? k0 + group : K;
        float a0 = 0.0f, a1 = 0.0f;
        for (int64_t k = k0; k < k1; ++k) {
            const int b = Q[k * ldq + c];
            const float v = to_f32(x[k]);
            bad |= !isfinite(v);
            a0 = fmaf(v, (float)((b << 28) >> 28), a0);
            a1 = fmaf(v, (float)((b << 24) >> 28), a1);
        }
        y0 = fmaf(a0, scale[g * lds + 2 * c], y0);
        if (two) y1 = fmaf(a1, scale[g * lds + 2 * c + 1], y1);
    }
    if (bad) set_status(dstatus, BSG_DSTATUS_NONFINITE);
    T *y = Y + blockIdx.y * ldy + 2 * c;
    y[0] = from_f32<T>(relu && !(y0 > 0.0f) ? 0.0f : y0);
    if (two) y[1] = from_f32<T>(relu && !(y1 > 0.0f) ? 0.0f : y1);
}

}  // namespace

cudaError_t launch_wquant_groups(const float *W, int64_t K, int64_t N, int64_t ldw, int64_t group,
                                 uint8_t *Q, int64_t ldq, float *scale, int64_t lds,
                                 int32_t *dstatus, cudaStream_t st) {
    const int64_t groups = (K + group - 1) / group;
    const dim3 grid((unsigned)(((N + 1) / 2 + 127) / 128),
                    (unsigned)(groups < 65535 ? groups : 65535));
    wquant_groups_kernel<<<grid, 128, 0, st>>>(W, K, N, ldw, group, Q, ldq, scale, lds, dstatus);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_wgroups_matvec(const void *X, int dtype, int64_t ldx, const uint8_t *Q,
                                  int64_t ldq, const float *scale, int64_t lds, int64_t group,
                                  int64_t M, int64_t N, int64_t K, int relu, void *Y, int64_t ldy,
                                  int32_t *dstatus, cudaStream_t st) {
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const dim3 grid((unsigned)(((N + 1) / 2 + 127) / 128), (unsigned)M);
        wgroups_matvec_kernel<T><<<grid, 128, 0, st>>>((const T *)X, ldx, Q, ldq, scale, lds,
                                                       group, N, K, relu, (T *)Y, ldy, dstatus);
        count_launches(1);
        return cudaGetLastError();
    });
}

}  // namespace bsg
