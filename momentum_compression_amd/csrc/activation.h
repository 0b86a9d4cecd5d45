// The activations of a product's epilogue and their slopes, in binary32.
#pragma once

#include "common.h"

namespace onebit {

__device__ __forceinline__ float exp_of(float x) {
    return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

// 1 / (1 + exp(-x)); the exponential's infinity gives 0.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + exp_of(-x));
}

// The normal distribution's integral from |z| on, and e^(-z^2 / 2).  The integral over
// the exponential is t P(t), t = 1 / (1 + p |z|), with P fitted in binary64 (weighted
// least squares towards the least largest error, |z| up to 13) so that the product is off
// by 3e-8 at most and by 4e-6 of itself: a small tail keeps its size.  In binary32 1.6e-7
// and 1.5e-5 of itself, the latter from the exponential's argument.
__device__ __forceinline__ float normal_tail(float z, float& bell) {
    const float s = z * 0.84932180028801904f;  // s^2 = z^2 log2(e) / 2
    bell = __builtin_amdgcn_exp2f(-s * s);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.34648234f, __builtin_fabsf(z), 1.0f));
    float p = __builtin_fmaf(0.044449616f, t, -0.18896839f);
    p = __builtin_fmaf(p, t, 0.22724105f);
    p = __builtin_fmaf(p, t, -0.0024435115f);
    p = __builtin_fmaf(p, t, 0.14663193f);
    p = __builtin_fmaf(p, t, 0.13465841f);
    p = __builtin_fmaf(p, t, 0.13843092f);
    return p * (t * bell);
}

constexpr float kTanhRate = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// z times a share that is 0 from -kNothing on: the limit there is 0 (z itself
// goes into the share, so a NaN stays one).
constexpr float kNothing = 200.0f;
__device__ __forceinline__ float share_of(float z, float share) {
    return fmaxf(z, -kNothing) * share;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if (ACT == ONEBIT_RELU) return z > 0.0f || z != z ? z : 0.0f;
    if (ACT == ONEBIT_GELU) {
        // z Phi(z) of either sign; the tail of a NaN is one
        float bell;
        const float tail = normal_tail(z, bell);
        return __builtin_fmaf(-fminf(__builtin_fabsf(z), kNothing), tail, fmaxf(z, 0.0f));
    }
    // 0.5 (1 + tanh u) = sigmoid(2 u)
    if (ACT == ONEBIT_GELU_TANH)
        return share_of(z, sigmoid(kTanhRate * __builtin_fmaf(kTanhCubic * z * z, z, z)));
    if (ACT == ONEBIT_SILU) return share_of(z, sigmoid(z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float slope(float z) {
    if (ACT == ONEBIT_RELU) return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    // what multiplies z is 0 long before +-kNothing
    const float near = fminf(fmaxf(z, -kNothing), kNothing);
    if (ACT == ONEBIT_GELU) {
        float bell;
        const float tail = normal_tail(z, bell);
        return __builtin_fmaf(near * bell, 0.39894228040143268f, z < 0.0f ? tail : 1.0f - tail);
    }
    if (ACT == ONEBIT_GELU_TANH) {
        const float s = sigmoid(kTanhRate * __builtin_fmaf(kTanhCubic * z * z, z, z));
        const float rate = kTanhRate * __builtin_fmaf(3.0f * kTanhCubic * near, near, 1.0f);
        return __builtin_fmaf(near * (s * (1.0f - s)), rate, s);
    }
    if (ACT == ONEBIT_SILU) {
        const float s = sigmoid(z);
        return __builtin_fmaf(near, s * (1.0f - s), s);
    }
    return 1.0f;
}

}  // namespace onebit
