// serve.cuh -- what the serving kernels share: activation types, the scale
// and code of a value, and status bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsgemm.h"

namespace bsg {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// The cache's scale of an absmax, one product where the unit of rows has a
// quotient: by this operator's definition, and at times a last place beside the unit's,
// so that a page's codes need not be the unit's of the same block (they stay within
// +-127: m / s <= 127 (1 + 2^-22)).
__device__ __forceinline__ float kv8_scale(float absmax) {
    return fmaxf(__fmul_rn(absmax, 1.0f / 127.0f), 1e-8f);
}
// The unit's code floor(RN(RN(x inv) + 0.5)) in the low byte; a non-finite x gives
// some byte.  Added to 1.5 2^23, where floats are the whole numbers, and rounded
// down, y is its floor, in the sum's low bits.
__device__ __forceinline__ uint32_t unit_code(float x, float inv) {
    return __float_as_uint(__fadd_rd(__fadd_rn(__fmul_rn(x, inv), 0.5f), 12582912.0f));
}

__device__ __forceinline__ void set_status(int32_t *dstatus, int32_t bits) {
    if (dstatus && bits) atomicOr(dstatus, bits);
}

// f(T{}) with the C++ type T of a bsg_dtype.
template <typename F>
cudaError_t with_dtype(int dtype, F &&f) {
    switch (dtype) {
        case BSG_F32: return f(float{});
        case BSG_F16: return f(__half{});
        default: return f(__nv_bfloat16{});
    }
}

}  // namespace
}  // namespace bsg
