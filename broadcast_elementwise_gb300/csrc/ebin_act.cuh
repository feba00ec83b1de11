// The activations of a product's epilogue and their derivatives, in binary32.
//
// 16-bit data takes fast forms, whose error is small against the 2^-8 or 2^-11 of
// the rounding that follows, relative to the result, its tails included: the
// hardware's 2^x and 1/x, and the normal distribution's lower tail as
//     Phi(-a) = (c1 t + .. + c6 t^6) exp(-a^2 / 2),  t = 1 / (1 + p a),  a >= 0,
// the form of 7.1.26 in Abramowitz and Stegun's Handbook of Mathematical Functions
// with p and the c fitted here to the quotient of both sides (Lawson's weighted
// least squares, a in [0, 13.2], past which the exponential is 0): off by 1.4e-7 at
// most, and by 2.6e-5 of Phi(-a) at most.  binary32 data takes the full ones
// (Phi by erff: a few 2^-24 of 1).
#pragma once

#include "ebin_layer.h"

namespace ebin {

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float act_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float act_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float act_sigmoid(float z) {
    return act_rcp(1.0f + act_ex2(-kLog2e * z));
}
constexpr float kPhiP = 0.295122355f;
constexpr float kPhi1 = 0.118483394f, kPhi2 = 0.107596874f, kPhi3 = 0.161231399f,
                kPhi4 = -0.0550026745f, kPhi5 = 0.251741707f, kPhi6 = -0.0840508044f;
// Phi(z)
__device__ __forceinline__ float act_normal(float z) {
    const float e = act_ex2(z * z * (-0.5f * kLog2e));
    const float t = act_rcp(fmaf(fabsf(z), kPhiP, 1.0f));
    float q = fmaf(t, kPhi6, kPhi5);
    q = fmaf(q, t, kPhi4);
    q = fmaf(q, t, kPhi3);
    q = fmaf(q, t, kPhi2);
    q = fmaf(q, t, kPhi1) * t * e;
    return z < 0.0f ? q : 1.0f - q;
}
__device__ __forceinline__ float act_tanh_arg(float z) {   // 2 sqrt(2/pi) (z + 0.044715 z^3)
    return z * fmaf(z * z, 0.0713548162726f, 1.59576912161f);
}

// The activation, for 16-bit data.
template <int ACT> __device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == EBIN_ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays
    if constexpr (ACT == EBIN_ACT_GELU) return z * act_normal(z);
    // (1 + tanh u) / 2 = sigmoid(2 u)
    if constexpr (ACT == EBIN_ACT_GELU_TANH) return z * act_sigmoid(act_tanh_arg(z));
    if constexpr (ACT == EBIN_ACT_SILU) return z * act_sigmoid(z);
    return z;
}

// Derivatives are flat, 0 or 1, far out and up to an infinite z (which a binary16
// pre-activation past 65504 is stored as).  Past kActFar every exponential below is 0
// or infinite, so z is held to it: the formulas would multiply an infinite z by 0.
constexpr float kActFar = 100.0f;

// A NaN stays one.  binary32, then 16-bit z alone and two to a word.
__device__ __forceinline__ float act_near(float z) {
    asm("max.NaN.f32 %0, %0, %1;\n\tmin.NaN.f32 %0, %0, %2;" : "+f"(z) : "f"(-kActFar), "f"(kActFar));
    return z;
}
template <class T> __device__ __forceinline__ T act_near(T z) {
    return __hmin_nan(__hmax_nan(z, from_f<T>(-kActFar)), from_f<T>(kActFar));
}
template <class T> __device__ __forceinline__ uint32_t act_near2(uint32_t w) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                         __nv_bfloat162>::type;
    T2 lo, hi;
    lo.x = lo.y = from_f<T>(-kActFar);
    hi.x = hi.y = from_f<T>(kActFar);
    const T2 z = __hmin2_nan(__hmax2_nan(*reinterpret_cast<const T2 *>(&w), lo), hi);
    return *reinterpret_cast<const uint32_t *>(&z);
}

// The derivative in full binary32, |z| <= kActFar.
template <int ACT> __device__ __forceinline__ float act_slope_full(float z) {
    if constexpr (ACT == EBIN_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == EBIN_ACT_GELU)
        return fmaf(z * 0.398942280401f, expf(-0.5f * z * z),
                    0.5f * (1.0f + erff(z * 0.707106781187f)));
    if constexpr (ACT == EBIN_ACT_GELU_TANH) {
        const float s = 1.0f / (1.0f + expf(-act_tanh_arg(z)));
        const float du = fmaf(z * z, 0.214064448818f, 1.59576912161f);
        return fmaf(z * (s * (1.0f - s)), du, s);
    }
    if constexpr (ACT == EBIN_ACT_SILU) {
        const float s = 1.0f / (1.0f + expf(-z));
        return fmaf(z, s * (1.0f - s), s);
    }
    return 1.0f;
}

__device__ __forceinline__ float2 act_pair(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 act_ex2(float2 x) {
    return make_float2(act_ex2(x.x), act_ex2(x.y));
}
__device__ __forceinline__ float2 act_rcp(float2 x) {
    return make_float2(act_rcp(x.x), act_rcp(x.y));
}

// The derivative for 16-bit data, |z| <= kActFar, two at a time on the packed
// binary32 pipe.
template <int ACT> __device__ __forceinline__ float2 act_slope2(float2 z) {
    if constexpr (ACT == EBIN_ACT_RELU)
        return make_float2(act_slope_full<ACT>(z.x), act_slope_full<ACT>(z.y));
    if constexpr (ACT == EBIN_ACT_GELU) {
        const float2 zz = __fmul2_rn(z, z);
        const float2 e = act_ex2(__fmul2_rn(zz, act_pair(-0.5f * kLog2e)));
        const float2 t = act_rcp(__ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)),
                                            act_pair(kPhiP), act_pair(1.0f)));
        float2 q = __ffma2_rn(t, act_pair(kPhi6), act_pair(kPhi5));
        q = __ffma2_rn(q, t, act_pair(kPhi4));
        q = __ffma2_rn(q, t, act_pair(kPhi3));
        q = __ffma2_rn(q, t, act_pair(kPhi2));
        q = __ffma2_rn(q, t, act_pair(kPhi1));
        q = __fmul2_rn(__fmul2_rn(q, t), e);
        const float2 up = make_float2(z.x < 0.0f ? q.x : 1.0f - q.x, z.y < 0.0f ? q.y : 1.0f - q.y);
        return __ffma2_rn(__fmul2_rn(z, act_pair(0.39894228f)), e, up);
    }
    if constexpr (ACT == EBIN_ACT_GELU_TANH) {
        const float2 zz = __fmul2_rn(z, z);
        const float2 u = __fmul2_rn(
            z, __ffma2_rn(zz, act_pair(0.0713548163f), act_pair(1.59576912f)));
        const float2 s = act_rcp(
            __fadd2_rn(act_ex2(__fmul2_rn(u, act_pair(-kLog2e))), act_pair(1.0f)));
        const float2 t = __ffma2_rn(make_float2(-s.x, -s.y), s, s);
        const float2 du = __ffma2_rn(zz, act_pair(0.214064449f), act_pair(1.59576912f));
        return __ffma2_rn(__fmul2_rn(z, t), du, s);
    }
    if constexpr (ACT == EBIN_ACT_SILU) {
        const float2 s = act_rcp(
            __fadd2_rn(act_ex2(__fmul2_rn(z, act_pair(-kLog2e))), act_pair(1.0f)));
        const float2 t = __ffma2_rn(make_float2(-s.x, -s.y), s, s);
        return __ffma2_rn(z, t, s);
    }
    return act_pair(1.0f);
}

}  // namespace ebin
