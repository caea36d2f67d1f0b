// recurrence_math.cuh -- one element of the gated channel recurrence (recurrence.cu), in fp32:
//   g = g_min s(e^A z),  h_t = e^g h_{t-1} + sqrt(1 - e^{2g}) s(i) x,  s the logistic function.
// The decay is kept as c = e^g - 1: a channel that remembers for thousands of tokens has a decay
// next to one, whose rounding to fp32 would be a relative error of the memory's length, and the
// input's factor m = sqrt(1 - e^{2g}) = sqrt(-c (2 + c)) has no cancellation in it.
#pragma once

#include "kda_common.cuh"

namespace kda {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// e^g - 1 for g <= 0.  Near zero by the series (its first left-out term is 5e-8 of the sum at
// -1/4); below, 1 is at least 4 times what e^g's rounding can lose (5e-7 of the result).
__device__ __forceinline__ float expm1_neg(float g) {
    float p = fmaf(g, 1.f / 720, 1.f / 120);
    p = fmaf(g, p, 1.f / 24);
    p = fmaf(g, p, 1.f / 6);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g, p, 1.f);
    return g > -0.25f ? g * p : ex2_approx(g * kLog2e) - 1.f;
}

// Per channel: what turns z into exponents of two, and e^A itself.
struct ChannelRate {
    float rate;      // e^A
    float neg_log2;  // -e^A log2(e)
};
__device__ __forceinline__ ChannelRate channel_rate(float A_log) {
    const float r = expf(A_log);
    return ChannelRate{r, -r * kLog2e};
}

// c and the input term b of one element.
struct Step {
    float c, b;
};
__device__ __forceinline__ Step recurrence_step(float x, float z, float i, float neg_log2,
                                                float g_min) {
    const float sz = rcp_approx(1.f + ex2_approx(z * neg_log2));
    const float si = rcp_approx(1.f + ex2_approx(-kLog2e * i));
    const float c = expm1_neg(g_min * sz);
    const float m2 = -c * (2.f + c);
    // (below 1e-37 the root would be of a denormal number: the factor is then zero)
    const float m = m2 > 1e-37f ? m2 * rsqrt_approx(m2) : m2 * 0.f;
    return Step{c, m * (si * x)};
}
// h_t from h_{t-1}
__device__ __forceinline__ float recurrence_next(float c, float b, float h) {
    return h + fmaf(c, h, b);
}

// c, and the factors of l_t = dL/dh_t in the gradients of one element, for the state h before it
// (that of dx is b / x).
struct StepGrad {
    float c, dx, di, dz;
};
__device__ __forceinline__ StepGrad recurrence_grad(float x, float z, float i, float rate,
                                                    float neg_log2, float g_min, float h) {
    // (limited, so that 1 - s = e^{-..} s stays a number where s is zero)
    const float ez = ex2_approx(z * neg_log2), ei = ex2_approx(-kLog2e * i);
    const float sz = rcp_approx(1.f + ez), si = rcp_approx(1.f + ei);
    const float oz = fminf(ez, 3e38f) * sz, oi = fminf(ei, 3e38f) * si;
    const float g = g_min * sz;
    const float c = expm1_neg(g), a = 1.f + c;
    const float m2 = -c * (2.f + c);
    const float q = m2 > 1e-37f ? rsqrt_approx(m2) : m2 * 0.f;  // 1 / m
    const float u = si * x;
    StepGrad r;
    r.c = c;
    r.dx = m2 * q * si;
    r.di = m2 * q * u * oi;
    r.dz = rate * oz * g * a * (h - a * q * u);
    return r;
}

}  // namespace kda
