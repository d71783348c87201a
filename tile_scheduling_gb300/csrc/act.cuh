// Activations of a linear layer and their slopes, in fp32.
//
//   relu max(z, 0);  gelu z Phi(z);  gelu_tanh z sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3), which is
//   z (1 + tanh u) / 2;  silu z sigmoid(z)
//
// sigmoid is formed as 1 / (1 + e^-z) with the fast exponential and division: each is good to
// 2 units in the last place near its argument, the exponent's rounding adds 2^-24 |z|, and an
// overflow to infinity gives the right limit 0.  A NaN stays one.
#pragma once
#include "linear_params.h"

namespace ts {

__device__ __forceinline__ float sigmoid_f32(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.f ? 0.f : z;
    if constexpr (ACT == ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid_f32(1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f));
    if constexpr (ACT == ACT_SILU) return z * sigmoid_f32(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.f ? 1.f : (z == z ? 0.f : z);
    if constexpr (ACT == ACT_GELU)
        return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), 0.5f * (1.f + erff(z * 0.70710678118654752f)));
    if constexpr (ACT == ACT_GELU_TANH) {
        const float s = sigmoid_f32(1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f));
        // 2 u' z; beyond |z| = 16 the factor s (1 - s) is 0, and the bound keeps the other one finite
        const float b = fminf(fmaxf(z, -16.f), 16.f);
        return fmaf(s * (1.f - s), 1.5957691216057308f * b * fmaf(0.134145f * b, b, 1.f), s);
    }
    if constexpr (ACT == ACT_SILU) {
        const float s = sigmoid_f32(z);
        return s * fmaf(z, 1.f - s, 1.f);
    }
    return 1.f;
}

// f(ACT as a type) for the activation chosen at run time.
template <int A>
struct ActTag {
    static constexpr int value = A;
};
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
        case ACT_RELU: f(ActTag<ACT_RELU>{}); break;
        case ACT_GELU: f(ActTag<ACT_GELU>{}); break;
        case ACT_GELU_TANH: f(ActTag<ACT_GELU_TANH>{}); break;
        case ACT_SILU: f(ActTag<ACT_SILU>{}); break;
        default: break;
    }
}

}  // namespace ts
