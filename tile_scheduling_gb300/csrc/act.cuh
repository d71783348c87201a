// Activations of a linear layer and their slopes, in fp32.
//
//   relu max(z, 0);  gelu z Phi(z);  gelu_tanh z sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3), which is
//   z (1 + tanh u) / 2;  silu z sigmoid(z)
//
// sigmoid is formed as 1 / (1 + e^-z) with the fast exponential and division: each is good to
// 2 units in the last place near its argument, the exponent's rounding adds 2^-24 |z|, and an
// overflow to infinity gives the right limit 0.  A NaN stays one.
//
// Phi uses Hastings' approximation of the error function (Abramowitz and Stegun, Handbook of
// Mathematical Functions, 7.1.26), which is off by at most 1.5e-7, about as much as fp32 itself
// near 1; its exponential is the one that the slope needs as well.  (With erff the gradient of
// 8192 x 8192 bf16 values took 123 us.)
#pragma once
#include "linear_params.h"

namespace ts {

__device__ __forceinline__ float sigmoid_f32(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// Phi(z), and exp(-z^2 / 2) on the way
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float t = __fdividef(1.f, fmaf(0.23164188f, fabsf(z), 1.f));  // 0.3275911 / sqrt(2)
    e = __expf(-0.5f * z * z);
    const float tail = 0.5f * e * t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
    return z < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.f ? 0.f : z;
    if constexpr (ACT == ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid_f32(1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f));
    if constexpr (ACT == ACT_SILU) return z * sigmoid_f32(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.f ? 1.f : (z == z ? 0.f : z);
    if constexpr (ACT == ACT_GELU) {
        float e;
        const float c = normal_cdf(z, e);
        return fmaf(z * 0.39894228040143268f, e, c);
    }
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
