// wq_round.cuh -- the weight storage's rounding: the integer nearest the exact
// quotient w / s, ties to even, without an f32 or f64 divide per element.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace bsg {
namespace {

// The integer nearest w / s, ties to even, clamped to [-qmax, qmax]; w and s
// finite, s > 0.  With w = mw 2^(ew-150) and s = ms 2^(es-150) (significands
// with the implicit bit; subnormals take exponent field 1 and no implicit
// bit), 2|w|/s = mw 2^sh / ms with sh = ew - es + 1, a ratio of integers.
__device__ __forceinline__ int wq_round_quotient_exact(float w, float s, int qmax) {
    const uint32_t wb = __float_as_uint(w);
    const uint32_t aw = wb & 0x7fffffffu;
    const int neg = (int)(wb >> 31);
    if (aw == 0) return 0;
    const uint32_t sb = __float_as_uint(s);
    const int ew = (int)(aw >> 23), es = (int)(sb >> 23);
    const uint64_t mw = (aw & 0x7fffffu) | (ew ? 0x800000u : 0u);
    const uint64_t ms = (sb & 0x7fffffu) | (es ? 0x800000u : 0u);
    const int sh = (ew ? ew : 1) - (es ? es : 1) + 1;
    // sh <= -25: 2|w|/s < 2^24 2^-25 = 1/2, so |w|/s < 1/4 and the code is 0;
    // sh >= 33: 2|w|/s > 2^33 / 2^24 = 512, beyond any qmax
    if (sh <= -25) return 0;
    if (sh >= 33) return neg ? -qmax : qmax;
    const uint64_t num = sh >= 0 ? mw << sh : mw;          // < 2^56
    const uint64_t den = sh >= 0 ? ms : ms << (-sh);        // < 2^48
    if (num >= (uint64_t)(2 * qmax + 2) * den) return neg ? -qmax : qmax;  // |w|/s >= qmax + 1
    // q2 = floor(2|w|/s) <= 2 qmax + 1: a float estimate, corrected exactly
    uint32_t q2 = (uint32_t)__fdividef((float)num, (float)den);
    if ((uint64_t)q2 * den > num) --q2;
    if ((uint64_t)(q2 + 1) * den <= num) ++q2;
    const uint64_t rem = num - (uint64_t)q2 * den;
    uint32_t q = q2 >> 1;                                   // |w|/s = q + (q2 odd) / 2 + rem / (2 den)
    if (q2 & 1) q += (rem != 0 || (q & 1)) ? 1u : 0u;       // above a half: up; on it: to even
    if ((int)q > qmax) q = (uint32_t)qmax;
    return neg ? -(int)q : (int)q;
}

// The same integer, first from x = RN(w * r) with r = RN(1 / s) (one
// reciprocal per column instead of a divide per element): x is within
// |w/s| 2^-23 of the exact quotient (two roundings of 2^-24; r is a normal
// float, since s <= FLT_MAX / 7 < 2^126), below 2^-16 while |x| < 128, so
// when x lies more than 2^-14 from the nearest half-integer h, the exact
// quotient lies on the same side of h and rounds to rint(x).  (x - h is
// exact there: for |x| >= 1, x and h are within a factor of two; below,
// h = +-1/2 and |x - h| >= 1/4 unless |x| >= 1/4.)  Quotients near a
// half-integer, and any x that is not finite (r overflowing for a tiny s),
// take the exact path.
__device__ __forceinline__ bool wq_fast_code(float w, float r, int qmax, int &q) {
    const float x = __fmul_rn(w, r);
    if (!(fabsf(x) < 128.0f)) return false;
    const float h = __fadd_rn(floorf(x), 0.5f);
    if (!(fabsf(__fsub_rn(x, h)) > 0x1p-14f)) return false;
    q = (int)rintf(x);
    q = q < -qmax ? -qmax : (q > qmax ? qmax : q);
    return true;
}

__device__ __forceinline__ int wq_round_quotient(float w, float s, float r, int qmax) {
    int q;
    return wq_fast_code(w, r, qmax, q) ? q : wq_round_quotient_exact(w, s, qmax);
}

}  // namespace
}  // namespace bsg
