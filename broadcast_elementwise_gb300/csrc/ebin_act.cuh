// The activations of a product's epilogue and their derivatives, in binary32.
#pragma once

#include "ebin_layer.h"

namespace ebin {

// exp and the quotient are the fast forms (a few units of 2^-23, against the
// 2^-8 or 2^-11 of the rounding to 16 bits that follows).
__device__ __forceinline__ float act_sigmoid(float z) {
    return __fdividef(1.0f, 1.0f + __expf(-z));
}

__device__ __forceinline__ float act_tanh_arg(float z) {   // 2 sqrt(2/pi) (z + 0.044715 z^3)
    return z * fmaf(z * z, 0.0713548162726f, 1.59576912161f);
}

template <int ACT> __device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == EBIN_ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays
    if constexpr (ACT == EBIN_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.707106781187f));
    // (1 + tanh u) / 2 = sigmoid(2 u)
    if constexpr (ACT == EBIN_ACT_GELU_TANH) return z * act_sigmoid(act_tanh_arg(z));
    if constexpr (ACT == EBIN_ACT_SILU) return z * act_sigmoid(z);
    return z;
}

// The derivative.  FAST: with the fast forms of exp and the quotient, for
// 16-bit data; otherwise with the full ones (the result is kept in 32 bits).
template <bool FAST> __device__ __forceinline__ float act_exp(float x) {
    return FAST ? __expf(x) : expf(x);
}
template <bool FAST> __device__ __forceinline__ float act_over(float x) {
    return FAST ? __fdividef(1.0f, x) : 1.0f / x;
}
template <int ACT, bool FAST> __device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == EBIN_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == EBIN_ACT_GELU)
        return fmaf(z * 0.398942280401f, act_exp<FAST>(-0.5f * z * z),
                    0.5f * (1.0f + erff(z * 0.707106781187f)));
    if constexpr (ACT == EBIN_ACT_GELU_TANH) {
        const float s = act_over<FAST>(1.0f + act_exp<FAST>(-act_tanh_arg(z)));
        const float du = fmaf(z * z, 0.214064448818f, 1.59576912161f);
        const float t = s * (1.0f - s);
        return t == 0.0f ? s : fmaf(z * t, du, s);   // flat far out, where z du may be infinite
    }
    if constexpr (ACT == EBIN_ACT_SILU) {
        const float s = act_over<FAST>(1.0f + act_exp<FAST>(-z));
        const float t = s * (1.0f - s);
        return t == 0.0f ? s : fmaf(z, t, s);
    }
    return 1.0f;
}

}  // namespace ebin
