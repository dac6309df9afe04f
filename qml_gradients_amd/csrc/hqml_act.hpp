// Element types of the dense layer and its activations with their slopes.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/hqml.h"

namespace hqml {

struct bf16 {
    uint16_t u;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __builtin_bit_cast(float, (uint32_t)x.u << 16); }
__device__ __forceinline__ void narrow(float x, float &o) { o = x; }
// round to nearest even; a NaN stays one
__device__ __forceinline__ void narrow(float x, bf16 &o) { o.u = __builtin_bit_cast(uint16_t, (__bf16)x); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2).  With t = 1 / (1 + 0.3 |z|),
// Phi(-|z|) exp(z^2 / 2) / t is smooth in t on (0, 1]; the polynomial is its least largest relative
// error there, 1.5e-7 (weighted least squares, reweighted to the largest error).  Relative error of
// the tail, measured: 6e-7 down to z = -2, then growing with z^2 as the exponent's rounding does:
// 8e-7 at -4, 2.6e-6 at -8, 7.6e-6 at -12.  An eighth of erff and expf's instructions.
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    const float a = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, a, 1.0f));
    e = __builtin_amdgcn_exp2f(a * a * -0.72134752f);
    float p = 0.0356756443f;
    p = __builtin_fmaf(p, t, -0.157206790f);
    p = __builtin_fmaf(p, t, 0.206360008f);
    p = __builtin_fmaf(p, t, -0.0536897052f);
    p = __builtin_fmaf(p, t, 0.128564859f);
    p = __builtin_fmaf(p, t, 0.0999125095f);
    p = __builtin_fmaf(p, t, 0.120754113f);
    p = __builtin_fmaf(p, t, 0.119629289f);
    const float q = p * t * e;
    return z < 0.0f ? q : 1.0f - q;
}

// 1 / (1 + exp(-z)) and tanh.  FAST, for results held in bf16: the hardware's exp2 and reciprocal, good to
// (1 + |z|) 2^-23 or so against bf16's 2^-8.
template <bool FAST>
__device__ __forceinline__ float logistic(float z)
{
    if (FAST) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
    return 1.0f / (1.0f + expf(-z));
}

template <bool FAST>
__device__ __forceinline__ float tanh_of(float z)
{
    if (!FAST) return tanhf(z);
    // near 0 the quotient would cancel: two more terms of the series, off by z^6 17/315 below 0.1
    const float s = z * z, near = z * __builtin_fmaf(s, __builtin_fmaf(s, 2.0f / 15.0f, -1.0f / 3.0f), 1.0f);
    const float far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * 2.88539008f));
    return s < 0.01f ? near : far;
}

// n values through one activation.
template <bool FAST, int n>
__device__ __forceinline__ void activate(float (&z)[n], int act)
{
    switch (act) {
    case HQML_ACT_RELU:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = z[k] < 0.0f ? 0.0f : z[k];
        break;
    case HQML_ACT_GELU:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            float e;
            z[k] *= normal_cdf(z[k], e);
        }
        break;
    case HQML_ACT_SILU:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] *= logistic<FAST>(z[k]);
        break;
    case HQML_ACT_TANH:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = tanh_of<FAST>(z[k]);
        break;
    case HQML_ACT_SIGMOID:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = logistic<FAST>(z[k]);
        break;
    default: break;
    }
}

// z becomes d act / dz.
template <bool FAST, int n>
__device__ __forceinline__ void slope(float (&z)[n], int act)
{
    switch (act) {
    case HQML_ACT_RELU:
#pragma unroll
        for (int k = 0; k < n; ++k) z[k] = z[k] > 0.0f ? 1.0f : 0.0f;
        break;
    case HQML_ACT_GELU:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            float e;
            const float f = normal_cdf(z[k], e);
            z[k] = f + z[k] * e * 0.39894228f;
        }
        break;
    case HQML_ACT_SILU:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float f = logistic<FAST>(z[k]);
            z[k] = f * (1.0f + z[k] * (1.0f - f));
        }
        break;
    case HQML_ACT_TANH:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float t = tanh_of<FAST>(z[k]);
            z[k] = 1.0f - t * t;
        }
        break;
    case HQML_ACT_SIGMOID:
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float f = logistic<FAST>(z[k]);
            z[k] = f * (1.0f - f);
        }
        break;
    default: break;
    }
}

}  // namespace hqml
