// The activations of the fused epilogue and their slopes, for the backward passes
// (linear.hip, checkpoint.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "dg.h"

namespace dg {
namespace {

// d act / d z in FP32.  exp2 and the reciprocal are the hardware's (1 ulp), Phi's tail is the
// rational fit of the forward epilogue (relative error 7e-8 before FP32's roundings, its
// e^(-z^2/2) shared with the density): errors of FP32's own size, which the bias
// gradient's sum averages.  With the device library's expf, erff and division the
// pass was bound by its arithmetic (8192 x 4096, GELU: 55 us against 45; 2304 x
// 2112, tanh form: 12.4 against 9.2).  A fit that keeps only the absolute error
// small (1.5e-7 of erf) has three terms fewer and is off by 1 % at z = -8: 43.7 us
// against 44.5.
// Past |z| = 16 the slopes are 0 or 1 to the last bit (SiLU: past 200 its tail is
// below FP32); z is cut there, so that no infinity meets a zero.  A NaN stays a NaN.
__device__ __forceinline__ float cut(float z, float far) { return z > far ? far : z < -far ? -far : z; }
__device__ __forceinline__ float logistic2(float x) {      // 1 / (1 + 2^-x)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x));
}
template <int ACT>
__device__ __forceinline__ float slope(float z, float& value) {       // and the activation, with the same functions
    if constexpr (ACT == DG_ACT_RELU) {
        value = z > 0.f ? z : z <= 0.f ? 0.f : z;
        return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    }
    if constexpr (ACT == DG_ACT_SILU) {
        const float c = cut(z, 200.f);
        const float s = logistic2(1.44269504f * c);
        value = z * s;
        return s * __builtin_fmaf(c, 1.f - s, 1.f);
    }
    if constexpr (ACT == DG_ACT_GELU) {
        const float c = cut(z, 16.f);
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.30405593f, __builtin_fabsf(c), 1.f));
        const float e = __builtin_amdgcn_exp2f(-0.72134752f * c * c);
        float y = __builtin_fmaf(t, 0.036534112f, -0.15392894f);
        y = __builtin_fmaf(t, y, 0.18981865f);
        y = __builtin_fmaf(t, y, -0.041117497f);
        y = __builtin_fmaf(t, y, 0.12256832f);
        y = __builtin_fmaf(t, y, 0.10271288f);
        y = __builtin_fmaf(t, y, 0.12215308f);
        const float tail = __builtin_fmaf(t, y, 0.12125936f) * t * e;       // Phi(-|z|)
        const float phi = c < 0.f ? tail : 1.f - tail;
        value = z * phi;
        return __builtin_fmaf(0.39894228f * c, e, phi);
    }
    if constexpr (ACT == DG_ACT_GELU_TANH) {
        const float c = cut(z, 16.f);
        const float s = logistic2(2.30220820f * c * __builtin_fmaf(0.044715f * c, c, 1.f));
        value = z * s;
        return __builtin_fmaf(c * s * (1.f - s), __builtin_fmaf(0.21406445f * c, c, 1.59576912f), s);
    }
    value = z;
    return 1.f;
}
template <int ACT>
__device__ __forceinline__ float slope(float z) {
    float value;
    return slope<ACT>(z, value);
}

}  // namespace
}  // namespace dg
