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

// The normal distribution's integral up to z and e^(-z^2 / 2).  Abramowitz and
// Stegun 7.1.26 gives erfc(x) = (a1 t + ... + a5 t^5) e^(-x^2), t = 1 / (1 + p x),
// to 1.5e-7 for x >= 0; the other side is 1 minus it, so small results keep
// their size.  Sixteen instructions where the library's erf takes forty.
__device__ __forceinline__ float normal_integral(float z, float& bell) {
    const float x = __builtin_fabsf(z) * 0.70710678118654752f;
    bell = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
    float p = __builtin_fmaf(1.061405429f, t, -1.453152027f);
    p = __builtin_fmaf(p, t, 1.421413741f);
    p = __builtin_fmaf(p, t, -0.284496736f);
    p = __builtin_fmaf(p, t, 0.254829592f);
    const float tail = 0.5f * p * t * bell;
    return z < 0.0f ? tail : 1.0f - tail;
}

constexpr float kTanhRate = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// z times a share that may be 0 where z is -infinity: the limit is 0.
__device__ __forceinline__ float share_of(float z, float share) {
    return z == -INFINITY ? 0.0f : z * share;
}

__device__ __forceinline__ float activate(float z, int32_t act) {
    float bell;
    switch (act) {
        case ONEBIT_RELU: return z > 0.0f || z != z ? z : 0.0f;
        case ONEBIT_GELU: return share_of(z, normal_integral(z, bell));
        // 0.5 (1 + tanh u) = sigmoid(2 u)
        case ONEBIT_GELU_TANH:
            return share_of(z, sigmoid(kTanhRate * __builtin_fmaf(kTanhCubic * z * z, z, z)));
        case ONEBIT_SILU: return share_of(z, sigmoid(z));
        default: return z;
    }
}

// Eight at once: one branch on the kind.
template <int ACT>
__device__ __forceinline__ void activate8_as(float z[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = activate(z[e], ACT);
}
__device__ __forceinline__ void activate8(float z[8], int32_t act) {
    switch (act) {
        case ONEBIT_RELU: return activate8_as<ONEBIT_RELU>(z);
        case ONEBIT_GELU: return activate8_as<ONEBIT_GELU>(z);
        case ONEBIT_GELU_TANH: return activate8_as<ONEBIT_GELU_TANH>(z);
        case ONEBIT_SILU: return activate8_as<ONEBIT_SILU>(z);
        default: return;
    }
}

__device__ __forceinline__ float slope(float z, int32_t act) {
    switch (act) {
        case ONEBIT_RELU: return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
        case ONEBIT_GELU: {
            float bell;
            const float share = normal_integral(z, bell);
            const float zb = bell == 0.0f ? 0.0f : z * bell;
            return __builtin_fmaf(zb, 0.39894228040143268f, share);
        }
        case ONEBIT_GELU_TANH: {
            const float s = sigmoid(kTanhRate * __builtin_fmaf(kTanhCubic * z * z, z, z));
            const float rest = s * (1.0f - s);
            const float rate = kTanhRate * __builtin_fmaf(3.0f * kTanhCubic * z, z, 1.0f);
            return rest == 0.0f ? s : __builtin_fmaf(z * rest, rate, s);
        }
        case ONEBIT_SILU: {
            const float s = sigmoid(z), rest = s * (1.0f - s);
            return rest == 0.0f ? s : __builtin_fmaf(z, rest, s);
        }
        default: return 1.0f;
    }
}

template <int ACT>
__device__ __forceinline__ void times_slope8_as(float d[8], const float z[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] *= slope(z[e], ACT);
}
__device__ __forceinline__ void times_slope8(float d[8], const float z[8], int32_t act) {
    switch (act) {
        case ONEBIT_RELU: return times_slope8_as<ONEBIT_RELU>(d, z);
        case ONEBIT_GELU: return times_slope8_as<ONEBIT_GELU>(d, z);
        case ONEBIT_GELU_TANH: return times_slope8_as<ONEBIT_GELU_TANH>(d, z);
        case ONEBIT_SILU: return times_slope8_as<ONEBIT_SILU>(d, z);
        default: return;
    }
}

}  // namespace onebit
