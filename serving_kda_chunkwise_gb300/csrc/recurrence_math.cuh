// recurrence_math.cuh -- an element (a pair of channels) of the gated channel recurrence, in fp32:
//   g = g_min s(e^A z),  h_t = e^g h_{t-1} + sqrt(1 - e^{2g}) s(i) x,  s the logistic function.
// The decay is kept as c = e^g - 1: a channel that remembers for thousands of tokens has a decay
// next to one, whose rounding to fp32 would be a relative error of the memory's length, and the
// input's factor m = sqrt(1 - e^{2g}) = sqrt(-c (2 + c)) has no cancellation in it.
//   c comes from g / 2^k in [-1.25, 0], k so that g_min's is: there (e^w - 1) / w is a polynomial of
// degree 6 (fitted at Chebyshev points, 1.9e-8 off relative), and e^{2w} - 1 = c (2 + c) doubles w.
// On the FMA pipes and for pairs, where the special function unit is what the logistic functions'
// exponentials and reciprocals and the root take already.
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
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_pair(float2 x) {
    return make_float2(ex2_approx(x.x), ex2_approx(x.y));
}
// 1 / (1 + e)
__device__ __forceinline__ float2 rcp1_pair(float2 e) {
    e = add2(e, both(1.f));
    return make_float2(rcp_approx(e.x), rcp_approx(e.y));
}

// The gate's lower bound: g_min, and g_min / 2^doublings in [-1.25, 0).
struct GateBound {
    float g_min, scaled;
    int doublings;
};
inline GateBound gate_bound(float g_min) {
    GateBound b{g_min, g_min, 0};
    for (; b.scaled < -1.25f; b.scaled *= 0.5f) ++b.doublings;
    return b;
}

// e^g - 1 for g = w 2^doublings, w in [-1.25, 0].
__device__ __forceinline__ float2 expm1_pair(float2 w, int doublings) {
    float2 p = fma2(w, both(1.1634889e-4f), both(1.2614741e-3f));
    p = fma2(w, p, both(8.2301879e-3f));
    p = fma2(w, p, both(4.1622911e-2f));
    p = fma2(w, p, both(1.6665773e-1f));
    p = fma2(w, p, both(4.9999931e-1f));
    p = fma2(w, p, both(1.f));
    float2 c = mul2(w, p);
    for (; doublings > 0; --doublings) c = fma2(c, c, add2(c, c));
    return c;
}

// Per pair of channels: what turns z into exponents of two (-e^A log2(e)), and e^A g_min.
struct ChannelRate {
    float2 neg_log2, rate_g;
};
__device__ __forceinline__ ChannelRate channel_rate(float2 A_log, float g_min) {
    const float2 r = make_float2(expf(A_log.x), expf(A_log.y));
    return ChannelRate{mul2(r, both(-kLog2e)), mul2(r, both(g_min))};
}

// c and the negated input term -b.
struct Step {
    float2 c, nb;
};
__device__ __forceinline__ Step recurrence_step(float2 x, float2 z, float2 i, float2 neg_log2,
                                                const GateBound& gb) {
    const float2 sz = rcp1_pair(ex2_pair(mul2(z, neg_log2)));
    const float2 si = rcp1_pair(ex2_pair(mul2(i, both(-kLog2e))));
    const float2 c = expm1_pair(mul2(sz, both(gb.scaled)), gb.doublings);
    const float2 d = fma2(c, c, add2(c, c));  // -m^2
    // (below 1e-37, where the root would be of a denormal number, the factor is next to nothing)
    const float2 q = make_float2(rsqrt_approx(fmaxf(-d.x, 1e-37f)), rsqrt_approx(fmaxf(-d.y, 1e-37f)));
    return Step{c, mul2(mul2(d, q), mul2(si, x))};
}
// h_t from h_{t-1}
__device__ __forceinline__ float2 recurrence_next(float2 c, float2 nb, float2 h) {
    return fma2(nb, both(-1.f), fma2(c, h, h));
}

// c, and the negated factors of l_t = dL/dh_t in the gradients, for the state h before the token
// (that of dx is -b / x).
struct StepGrad {
    float2 c, dx, di, dz;
};
__device__ __forceinline__ StepGrad recurrence_grad(float2 x, float2 z, float2 i,
                                                    const ChannelRate& r, const GateBound& gb,
                                                    float2 h) {
    const float2 ez = ex2_pair(mul2(z, r.neg_log2)), ei = ex2_pair(mul2(i, both(-kLog2e)));
    const float2 sz = rcp1_pair(ez), si = rcp1_pair(ei);
    // 1 - s = e^{-..} s, the exponential limited so that it stays a number where s is zero
    const float2 oz = mul2(make_float2(fminf(ez.x, 3e38f), fminf(ez.y, 3e38f)), sz);
    const float2 oi = mul2(make_float2(fminf(ei.x, 3e38f), fminf(ei.y, 3e38f)), si);
    StepGrad o;
    o.c = expm1_pair(mul2(sz, both(gb.scaled)), gb.doublings);
    const float2 d = fma2(o.c, o.c, add2(o.c, o.c));
    const float2 q = make_float2(rsqrt_approx(fmaxf(-d.x, 1e-37f)), rsqrt_approx(fmaxf(-d.y, 1e-37f)));
    const float2 a = add2(o.c, both(1.f)), m = mul2(d, q), u = mul2(si, x);
    o.dx = mul2(m, si);
    o.di = mul2(mul2(m, u), oi);
    // e^A g (1 - s(e^A z)) e^g (e^g / m s(i) x - h)
    o.dz = mul2(mul2(mul2(r.rate_g, sz), mul2(oz, a)), fma2(h, both(-1.f), mul2(a, mul2(q, u))));
    return o;
}

}  // namespace kda
