// The activations of the GEMM epilogues and of the activation gradient, in
// fp32. sigmoid(x) = 1 / (1 + 2^(-x log2 e)) takes the two MUFU instructions
// ex2.approx and rcp.approx, whose documented errors are 2 ulp and 1 ulp: the
// results are within a few 2^-23 of the formula (relative to z; GELU's tail is
// below), under the bf16 or FP8 rounding that follows. Their .ftz forms are one
// instruction each, where the others scale subnormals around it; only a sigmoid
// or an exponential below 2^-126 is flushed. Everything else runs on pairs
// (fma.rn.f32x2 and its like), which rounds each half as the scalar instruction
// would at half the instructions: the epilogues and the gradient are bound by
// issue before they are by MUFU.
//   ReLU       z < 0 ? 0 : z                       (NaN stays NaN)
//   GELU       z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2 = 1 - Phi(-z), and
//              for x >= 0 Phi(-x) = exp(-x^2 / 2) P(1 / (1 + c x)), the form of
//              7.1.26 in Abramowitz and Stegun's handbook. That formula's own
//              P, of degree 5, is good to 7.5e-8 absolutely, which is 0.4 % of
//              Phi(-5) and 1 % of Phi(-8). The slope Phi(z) + z phi(z) takes
//              it: there z phi(z) outweighs Phi by z^2, and the tail is off by
//              less than 3e-4 of itself. The activation takes a P of degree 6,
//              fitted here to the smaller of 6e-8 absolute and 1e-4 relative
//              error over x <= 14.5, so that the tail too keeps the precision
//              of its rounding (in the slope it would cost 3 %: 32768 x 4096
//              147.4 -> 152.0 us; in the product 1 %: 2048 x 4096 x 1024
//              16.1 -> 16.3)
//   GELU tanh  z (1 + tanh u) / 2 = z sigmoid(2 u),
//              u = sqrt(2 / pi) (z + 0.044715 z^3)
//   SiLU       z sigmoid(z)
#pragma once

#include "common.cuh"

namespace fp8lite {

inline bool valid_act(int a) { return a >= FP8_ACT_NONE && a <= FP8_ACT_SILU; }

// Two fp32 values in one 64-bit register pair.
using F2 = unsigned long long;

__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float v) { return f2(v, v); }
__device__ __forceinline__ void split(F2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 ex2_2(F2 x) {
    float a, b;
    split(x, a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2(a, b);
}
__device__ __forceinline__ F2 rcp2(F2 x) {
    float a, b;
    split(x, a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2(a, b);
}

// max that keeps a NaN.
__device__ __forceinline__ float at_least(float x, float lo) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;
// -2 log2(e) sqrt(2 / pi) and 0.044715 times it: sigmoid(2u) = 1 / (1 + 2^(z (k0 + k1 z^2)))
constexpr float kGeluT0 = -2.3022081985f;
constexpr float kGeluT1 = -0.1029432396f;

// Phi(z), the standard normal distribution function; e is exp(-z^2 / 2).
// TAIL: to a relative 1e-4 however small.
template <bool TAIL>
__device__ __forceinline__ F2 normal_cdf(F2 z, F2& e) {
    // c; for 7.1.26 0.3275911 / sqrt 2, and half of its a1 t + ... + a5 t^5 below
    const F2 t = rcp2(fma2(z & 0x7FFFFFFF7FFFFFFFull, f2(TAIL ? 0.292f : 0.23164189f), f2(1.0f)));
    e = ex2_2(mul2(mul2(z, z), f2(-0.5f * kLog2e)));
    F2 p;
    if (TAIL) {
        p = fma2(t, f2(-0.08670647f), f2(0.2705679f));
        p = fma2(t, p, f2(-0.07591453f));
        p = fma2(t, p, f2(0.17060119f));
        p = fma2(t, p, f2(0.10403046f));
        p = fma2(t, p, f2(0.11742138f));
    } else {
        p = fma2(t, f2(0.5307027145f), f2(-0.7265760135f));
        p = fma2(t, p, f2(0.7107068705f));
        p = fma2(t, p, f2(-0.142248368f));
        p = fma2(t, p, f2(0.127414796f));
    }
    const F2 q = mul2(mul2(t, p), e);
    float z0, z1, q0, q1, r0, r1;
    split(z, z0, z1);
    split(q, q0, q1);
    split(fma2(q, f2(-1.0f), f2(1.0f)), r0, r1);
    return f2(z0 < 0.0f ? q0 : r0, z1 < 0.0f ? q1 : r1);
}

// act(z). Below -100 every activation but ReLU is 0 in fp32: limiting z first
// gives that also at -inf, where the formula would multiply it by 0.
template <int ACT>
__device__ __forceinline__ F2 act_fwd(F2 z) {
    if (ACT == FP8_ACT_NONE) return z;
    float a, b;
    split(z, a, b);
    if (ACT == FP8_ACT_RELU) return f2(a < 0.0f ? 0.0f : a, b < 0.0f ? 0.0f : b);
    z = f2(at_least(a, -100.0f), at_least(b, -100.0f));
    if (ACT == FP8_ACT_GELU) {
        F2 e;
        return mul2(z, normal_cdf<true>(z, e));
    }
    const F2 x = ACT == FP8_ACT_GELU_TANH ? mul2(z, fma2(mul2(z, z), f2(kGeluT1), f2(kGeluT0))) : mul2(z, f2(-kLog2e));
    return mul2(z, rcp2(add2(ex2_2(x), f2(1.0f))));
}

// act'(z) of a pair of bf16 values, the first in the low half. z is limited
// to a range outside which the slope is 0 or 1 in fp32 (under 2^-100 off),
// so that 2^x below stays finite and infinities give the limits.
template <int ACT>
__device__ __forceinline__ F2 act_slope(uint32_t zz) {
    if (ACT == FP8_ACT_NONE) return f2(1.0f);
    if (ACT == FP8_ACT_RELU) {
        // s = z > 0 on the pair, and min(max(z, s), s): s again, but NaN where z is
        // (32768 x 4096: 105.4 us; 105.0 where a NaN gives 0, 107.6 by compares in fp32)
        uint32_t s;
        asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(s) : "r"(zz), "r"(0u));
        asm("max.NaN.bf16x2 %0, %0, %1;\n\tmin.NaN.bf16x2 %0, %0, %1;" : "+r"(zz) : "r"(s));
        return f2(__uint_as_float(zz << 16), __uint_as_float(zz & 0xFFFF0000u));
    }
    // bf16 pairs: 100; -10 (GELU tanh), -87 (SiLU), -100 (GELU)
    constexpr uint32_t kLo = ACT == FP8_ACT_GELU_TANH ? 0xC120C120u : ACT == FP8_ACT_SILU ? 0xC2AEC2AEu : 0xC2C8C2C8u;
    asm("max.NaN.bf16x2 %0, %0, %1;\n\tmin.NaN.bf16x2 %0, %0, %2;" : "+r"(zz) : "r"(kLo), "r"(0x42C842C8u));
    const float z0 = __uint_as_float(zz << 16), z1 = __uint_as_float(zz & 0xFFFF0000u);
    const F2 z = f2(z0, z1);
    if (ACT == FP8_ACT_GELU) {
        F2 e;
        const F2 c = normal_cdf<false>(z, e);
        return fma2(z, mul2(e, f2(0.3989422804f)), c);  // Phi + z phi
    }
    // y = z s: y' = s + s z (1 - s) w', where s = 1 / (1 + e) and 1 - s = e s (no cancellation)
    if (ACT == FP8_ACT_GELU_TANH) {
        const F2 zsq = mul2(z, z);
        const F2 e = ex2_2(mul2(z, fma2(zsq, f2(kGeluT1), f2(kGeluT0))));
        const F2 s = rcp2(add2(e, f2(1.0f)));
        // w' = 2 sqrt(2/pi) (1 + 3 * 0.044715 z^2), the derivative of 2u
        return fma2(s, mul2(mul2(z, mul2(e, s)), fma2(zsq, f2(0.2140644488f), f2(1.5957691216f))), s);
    }
    const F2 e = ex2_2(mul2(z, f2(-kLog2e)));
    const F2 s = rcp2(add2(e, f2(1.0f)));
    return fma2(s, mul2(z, mul2(e, s)), s);
}

template <int ACT, int N>
__device__ __forceinline__ void act_each(float (&y)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) split(act_fwd<ACT>(f2(y[i], y[i + 1])), y[i], y[i + 1]);
}

// One activation over the values of a register array; the choice is uniform
// over the launch, so it costs one branch per call.
template <int N>
__device__ __forceinline__ void act_apply(int act, float (&y)[N]) {
    if (act == FP8_ACT_RELU) act_each<FP8_ACT_RELU>(y);
    else if (act == FP8_ACT_GELU) act_each<FP8_ACT_GELU>(y);
    else if (act == FP8_ACT_GELU_TANH) act_each<FP8_ACT_GELU_TANH>(y);
    else if (act == FP8_ACT_SILU) act_each<FP8_ACT_SILU>(y);
}

}  // namespace fp8lite
