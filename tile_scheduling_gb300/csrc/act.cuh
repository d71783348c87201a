// Activations of a linear layer and their slopes, in fp32, two values at a time.
//
//   relu max(z, 0);  gelu z Phi(z);  gelu_tanh z sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3), which is
//   z (1 + tanh u) / 2;  silu z sigmoid(z)
//
// sigmoid is formed as 1 / (1 + e^-z) with the approximate base-2 exponential and reciprocal: each is
// good to 2 units in the last place, the exponent's rounding adds 2^-24 |z|, and an overflow to infinity
// gives the right limit 0.  A NaN stays one.
//
// Phi uses Hastings' approximation of the error function (Abramowitz and Stegun, Handbook of
// Mathematical Functions, 7.1.26), which is off by at most 1.5e-7, about as much as fp32 itself
// near 1; its exponential is the one that the slope needs as well.
//
// An exponential and a reciprocal are taken for each value, the rest two values to an instruction: 8192 x
// 8192 bf16 gradients through gelu 72 us, bound by memory (one value at a time 94, with erff 123).
#pragma once
#include "linear_params.h"

namespace ts {

// Two fp32 values in a register pair.
struct Two {
    uint64_t v;
};
__device__ __forceinline__ Two two(float lo, float hi) {
    Two t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(t.v) : "f"(lo), "f"(hi));
    return t;
}
__device__ __forceinline__ Two two(float both) { return two(both, both); }
__device__ __forceinline__ void split(Two t, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(t.v));
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
template <class F>
__device__ __forceinline__ Two each(Two t, F &&f) {
    float lo, hi;
    split(t, lo, hi);
    return two(f(lo), f(hi));
}
template <class F>
__device__ __forceinline__ Two each(Two t, Two u, F &&f) {
    float lo, hi, ulo, uhi;
    split(t, lo, hi);
    split(u, ulo, uhi);
    return two(f(lo, ulo), f(hi, uhi));
}
__device__ __forceinline__ Two exp2_of(Two t) {
    return each(t, [](float x) {
        float r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
        return r;
    });
}
__device__ __forceinline__ Two reciprocal(Two t) {
    return each(t, [](float x) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
        return r;
    });
}

constexpr float kLog2e = 1.44269504f;
constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// 1 / (1 + 2^t)
__device__ __forceinline__ Two logistic(Two t) { return reciprocal(exp2_of(t) + two(1.f)); }
// sigmoid(2 u) of gelu_tanh
__device__ __forceinline__ Two tanh_gate(Two z) {
    return logistic(z * fma(z * z, two(-kLog2e * kTanhScale * 0.044715f), two(-kLog2e * kTanhScale)));
}

// Phi(z), and exp(-z^2 / 2) on the way
__device__ __forceinline__ Two normal_cdf(Two z, Two &e) {
    const Two az = each(z, [](float x) { return fabsf(x); });
    const Two t = reciprocal(fma(az, two(0.23164188f), two(1.f)));  // 0.3275911 / sqrt(2)
    e = exp2_of(z * z * two(-0.5f * kLog2e));
    // half of Hastings' coefficients
    Two p = fma(t, two(0.5f * 1.061405429f), two(0.5f * -1.453152027f));
    p = fma(t, p, two(0.5f * 1.421413741f));
    p = fma(t, p, two(0.5f * -0.284496736f));
    p = fma(t, p, two(0.5f * 0.254829592f));
    const Two tail = p * t * e;
    const Two rest = fma(tail, two(-1.f), two(1.f));
    float z0, z1, t0, t1, r0, r1;
    split(z, z0, z1);
    split(tail, t0, t1);
    split(rest, r0, r1);
    return two(z0 < 0.f ? t0 : r0, z1 < 0.f ? t1 : r1);
}

template <int ACT>
__device__ __forceinline__ Two act_of(Two z) {
    if constexpr (ACT == ACT_RELU) return each(z, [](float x) { return x < 0.f ? 0.f : x; });
    if constexpr (ACT == ACT_GELU) {
        Two e;
        return z * normal_cdf(z, e);
    }
    if constexpr (ACT == ACT_GELU_TANH) return z * tanh_gate(z);
    if constexpr (ACT == ACT_SILU) return z * logistic(z * two(-kLog2e));
    return z;
}

template <int ACT>
__device__ __forceinline__ Two act_slope(Two z) {
    if constexpr (ACT == ACT_RELU) return each(z, [](float x) { return x > 0.f ? 1.f : (x == x ? 0.f : x); });
    if constexpr (ACT == ACT_GELU) {
        Two e;
        const Two c = normal_cdf(z, e);
        return fma(z * two(0.39894228040143268f), e, c);
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const Two s = tanh_gate(z);
        // 2 u' z; beyond |z| = 16 the factor s (1 - s) is 0, and the bound keeps the other one finite
        const Two b = each(z, [](float x) { return fminf(fmaxf(x, -16.f), 16.f); });
        const Two u = b * fma(b * b, two(kTanhScale * 0.134145f), two(kTanhScale));
        return fma(fma(s, s * two(-1.f), s), u, s);
    }
    if constexpr (ACT == ACT_SILU) {
        const Two s = logistic(z * two(-kLog2e));
        return s * fma(z, fma(s, two(-1.f), two(1.f)), two(1.f));
    }
    return two(1.f);
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
        default: f(ActTag<ACT_NONE>{}); break;
    }
}
// x[i] = act(x[i]), and x[i] *= act'(a[i]), for an even number of values
template <int ACT, int N>
__device__ __forceinline__ void apply_act(float (&x)[N]) {
    if constexpr (ACT != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < N; i += 2) split(act_of<ACT>(two(x[i], x[i + 1])), x[i], x[i + 1]);
    }
}
template <int ACT, int N>
__device__ __forceinline__ void apply_slope(float (&x)[N], const float (&a)[N]) {
    if constexpr (ACT != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            split(two(x[i], x[i + 1]) * act_slope<ACT>(two(a[i], a[i + 1])), x[i], x[i + 1]);
    }
}

}  // namespace ts
