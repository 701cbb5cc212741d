// The activations of the GEMM epilogues and of the activation gradient, in
// fp32. sigmoid(x) = 1 / (1 + 2^(-x log2 e)) takes the two MUFU instructions
// ex2.approx and rcp.approx, whose documented errors are 2 ulp and 1 ulp: the
// results are within a few 2^-23 of the formula (relative to z), far below
// the bf16 or FP8 rounding that follows.
//   ReLU       z < 0 ? 0 : z                       (NaN stays NaN)
//   GELU       z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2, erf by the
//              rational form 7.1.26 of Abramowitz and Stegun's handbook
//              (absolute error 1.5e-7)
//   GELU tanh  z (1 + tanh u) / 2 = z sigmoid(2 u),
//              u = sqrt(2 / pi) (z + 0.044715 z^3)
//   SiLU       z sigmoid(z)
#pragma once

#include "common.cuh"

namespace fp8lite {

inline bool valid_act(int a) { return a >= FP8_ACT_NONE && a <= FP8_ACT_SILU; }

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max / min that keep a NaN. Below -100 (and above 100) every activation here
// is 0 (z) and every slope 0 (1) in fp32: limiting z to that range first gives
// the limits also at infinities, where the formulas would multiply 0 by inf.
__device__ __forceinline__ float at_least(float x, float lo) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
    return y;
}

__device__ __forceinline__ float at_most(float x, float hi) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(hi));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;
// -2 log2(e) sqrt(2 / pi) and 0.044715 times it: sigmoid(2u) = 1 / (1 + 2^(z (k0 + k1 z^2)))
constexpr float kGeluT0 = -2.3022081985f;
constexpr float kGeluT1 = -0.1029432396f;

// Phi(z), the standard normal distribution function; e is exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float a = fabsf(z);
    const float t = rcp_approx(fmaf(a, 0.23164189f, 1.0f));  // 0.3275911 / sqrt 2
    e = ex2_approx(z * z * (-0.5f * kLog2e));
    // half of (a1 t + a2 t^2 + a3 t^3 + a4 t^4 + a5 t^5)
    const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5307027145f, -0.7265760135f), 0.7107068705f), -0.142248368f),
                             0.127414796f);
    const float q = p * e;
    return z < 0.0f ? q : 1.0f - q;
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
    if (ACT == FP8_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if (ACT != FP8_ACT_NONE) z = at_least(z, -100.0f);
    if (ACT == FP8_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    if (ACT == FP8_ACT_GELU_TANH) return z * rcp_approx(1.0f + ex2_approx(z * fmaf(z * z, kGeluT1, kGeluT0)));
    if (ACT == FP8_ACT_SILU) return z * rcp_approx(1.0f + ex2_approx(z * -kLog2e));
    return z;
}

// act'(z).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == FP8_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    // the lower limit keeps 2^x finite below: the slope there is under 2^-100 already
    z = at_most(at_least(z, ACT == FP8_ACT_GELU_TANH ? -10.0f : ACT == FP8_ACT_SILU ? -87.0f : -100.0f), 100.0f);
    if (ACT == FP8_ACT_GELU) {
        float e;
        const float c = normal_cdf(z, e);
        return fmaf(z, e * 0.3989422804f, c);  // Phi + z phi
    }
    // y = z s: y' = s + s z (1 - s) w', where s = 1 / (1 + e) and 1 - s = e s (no cancellation)
    if (ACT == FP8_ACT_GELU_TANH) {
        const float z2 = z * z;
        const float e = ex2_approx(z * fmaf(z2, kGeluT1, kGeluT0));
        const float s = rcp_approx(1.0f + e);
        // w' = 2 sqrt(2/pi) (1 + 3 * 0.044715 z^2), the derivative of 2u
        return fmaf(s, (z * (e * s)) * fmaf(z2, 0.2140644488f, 1.5957691216f), s);
    }
    if (ACT == FP8_ACT_SILU) {
        const float e = ex2_approx(z * -kLog2e);
        const float s = rcp_approx(1.0f + e);
        return fmaf(s, z * (e * s), s);
    }
    return 1.0f;
}

// One activation over the values of a register array; the choice is uniform
// over the launch, so it costs one branch per call.
template <int N>
__device__ __forceinline__ void act_apply(int act, float (&y)[N]) {
    if (act == FP8_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = act_fwd<FP8_ACT_RELU>(y[i]);
    } else if (act == FP8_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = act_fwd<FP8_ACT_GELU>(y[i]);
    } else if (act == FP8_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = act_fwd<FP8_ACT_GELU_TANH>(y[i]);
    } else if (act == FP8_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = act_fwd<FP8_ACT_SILU>(y[i]);
    }
}

}  // namespace fp8lite
