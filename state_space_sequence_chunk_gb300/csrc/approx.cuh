// approx.cuh -- exponentials and sigmoids from the hardware's fast ones (2^v off by 2^-22 of it at
// most, 1 / v by 2^-23), singly and in pairs.
#pragma once

#include "f32x2.cuh"

namespace ssd {

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
    float a, b;
    unpair(v, a, b);
    return pair(ex2(a), ex2(b));
}
__device__ __forceinline__ float max_nan(float a, float b) {    // a NaN stays one
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pair(a, a); }
// exp(v).  The product with log2(e) is rounded; its remainder is added back (log2(e) in
// two floats), so that the result is good to the exponential's own error also where v is large: without it
// the scan's delta, and with it an fp32 state, is off by 7e-8 of it for each of |v| (2 % of the forward pass's
// time).  v from -200 (every power from there on is 0) to 80.
constexpr float kLog2eLow = 1.925963033500e-8f;       // log2(e) - kLog2e
__device__ __forceinline__ float exp_in_range(float v) {
    const float p = v * kLog2e, e = ex2(p);
    return fmaf(e * 0.69314718f, fmaf(v, kLog2eLow, fmaf(v, kLog2e, -p)), e);
}
__device__ __forceinline__ f32x2 exp_in_range2(f32x2 v) {
    const f32x2 q = mul2(v, both(-kLog2e)), lo = fma2(v, both(kLog2eLow), fma2(v, both(kLog2e), q));
    float a, b;
    unpair(q, a, b);
    const f32x2 e = pair(ex2(-a), ex2(-b));
    return fma2(e, mul2(lo, both(0.69314718f)), e);
}
// exp(-|v|); a NaN stays one.
__device__ __forceinline__ float exp_neg_abs(float v) { return exp_in_range(max_nan(-fabsf(v), -200.f)); }
__device__ __forceinline__ f32x2 exp_neg_abs2(float a, float b) {
    return exp_in_range2(pair(max_nan(-fabsf(a), -200.f), max_nan(-fabsf(b), -200.f)));
}
// 1 / (1 + exp(-z)).  EXACT, for fp32 operands: with the exponential's remainder, good to 9 * 2^-24 of it for
// every z (3 % of a convolution's time, 1 % of a scan's).  Without, for bf16 operands, whose results are rounded
// to 2^-8: off by 1.2 * 2^-24 more for each of |z| (the fp32 sums over tokens, of dweight or dA, take over the
// terms' 4e-7 at |z| = 5); with it their convolution of 16384 tokens of 5120 channels takes 65 us
// instead of 59, its gradient 122 instead of 108, their scan 3 % more.
template <bool EXACT> __device__ __forceinline__ float sigmoid(float z) {
    if (!EXACT) return rcp(1.f + ex2(-z * kLog2e));
    const float e = exp_neg_abs(z), r = rcp(1.f + e);
    return z >= 0.f ? r : e * r;
}
template <bool EXACT> __device__ __forceinline__ f32x2 sigmoid2(f32x2 z) {
    float a, b;
    if (!EXACT) {
        unpair(mul2(z, both(-kLog2e)), a, b);
        unpair(add2(pair(ex2(a), ex2(b)), both(1.f)), a, b);
        return pair(rcp(a), rcp(b));
    }
    float c, d, z0, z1;
    unpair(z, z0, z1);
    const f32x2 e = exp_neg_abs2(z0, z1);
    unpair(add2(e, both(1.f)), a, b);
    const f32x2 r = pair(rcp(a), rcp(b));
    unpair(r, a, b);
    unpair(mul2(e, r), c, d);
    return pair(z0 >= 0.f ? a : c, z1 >= 0.f ? b : d);
}

}  // namespace ssd
