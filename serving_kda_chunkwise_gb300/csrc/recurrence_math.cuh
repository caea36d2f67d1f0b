// recurrence_math.cuh -- an element (a pair of channels) of the gated channel recurrence, in fp32:
//   g = g_min s(e^A z),  h_t = e^g h_{t-1} + sqrt(1 - e^{2g}) s(i) x,  s the logistic function.
// The decay is kept as c = e^g - 1: a channel that remembers for thousands of tokens has a decay
// next to one, whose rounding to fp32 would be a relative error of the memory's length, and the
// input's factor m = sqrt(1 - e^{2g}) = sqrt(-c (2 + c)) has no cancellation in it.
//   c comes from g / 2^k in [-1.25, 0], k so that g_min's is: there (e^w - 1) / w is a polynomial of
// degree 5 (fitted, 3.3e-7 off relative), and e^{2w} - 1 = c (2 + c) doubles w.
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
// Pairs of numbers in one instruction.
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_pair(float2 x) {
    return make_float2(ex2_approx(x.x), ex2_approx(x.y));
}
// 1 / (1 + e)
__device__ __forceinline__ float2 rcp1_pair(float2 e) {
    e = add_pair(e, both(1.f));
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

// e^w - 1 for w in [-1.25, 0].
__device__ __forceinline__ float2 expm1_near(float2 w) {
    float2 p = fma_pair(w, both(8.2454522e-4f), both(7.6172315e-3f));
    p = fma_pair(w, p, both(4.1230343e-2f));
    p = fma_pair(w, p, both(1.6654715e-1f));
    p = fma_pair(w, p, both(4.9998909e-1f));
    p = fma_pair(w, p, both(1.f));
    return mul_pair(w, p);
}
// e^{2w} - 1 from e^w - 1
__device__ __forceinline__ float2 twice(float2 c) { return fma_pair(c, c, add_pair(c, c)); }

// Per pair of channels: what turns z into exponents of two (-e^A log2(e)), and e^A g_min.
struct ChannelRate {
    float2 neg_log2, rate_g;
};
__device__ __forceinline__ ChannelRate channel_rate(float2 A_log, float g_min) {
    const float2 r = make_float2(expf(A_log.x), expf(A_log.y));
    return ChannelRate{mul_pair(r, both(-kLog2e)), mul_pair(r, both(g_min))};
}

// 1 / sqrt(-d).  (Below 1e-37, where the root would be of a denormal number, what is multiplied by it
// is next to nothing.)
__device__ __forceinline__ float2 rsqrt_pair(float2 d) {
    return make_float2(rsqrt_approx(fmaxf(-d.x, 1e-37f)), rsqrt_approx(fmaxf(-d.y, 1e-37f)));
}

// n tokens in steps that leave the tokens independent of each other: c[k], and the negated input
// terms nb[k] = -b.  in(which, k): input x, z or i (0, 1, 2) of token k.  summed(the sum of the s(e^A z)).
//   b = m s(i) x = m^2 x / sqrt(m^2 (1 + e^-i)^2): one root for m's and s(i)'s reciprocal.  (1e-37 next
// to m^2 keeps it from zero, so that the root of 0 times infinity is not taken; an m below 3e-19 is
// lost in it, and a s(i) below 2^-64 in the square's overflow.)
template <int n, typename In, typename Sum>
__device__ __forceinline__ void recurrence_steps(In&& in, float2 neg_log2, const GateBound& gb,
                                                 float2 (&c)[n], float2 (&nb)[n], Sum&& summed) {
    float2 sum;
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const float2 sz = rcp1_pair(ex2_pair(mul_pair(in(1, k), neg_log2)));
        sum = k == 0 ? sz : add_pair(sum, sz);
        c[k] = expm1_near(mul_pair(sz, both(gb.scaled)));
        nb[k] = add_pair(ex2_pair(mul_pair(in(2, k), both(-kLog2e))), both(1.f));
    }
    summed(sum);
    for (int j = gb.doublings; j > 0; --j)
#pragma unroll
        for (int k = 0; k < n; ++k) c[k] = twice(c[k]);
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const float2 d = twice(c[k]);  // -m^2
        const float2 y = mul_pair(mul_pair(add_pair(d, both(-1e-37f)), nb[k]), nb[k]);
        const float2 q = make_float2(rsqrt_approx(-y.x), rsqrt_approx(-y.y));
        nb[k] = mul_pair(mul_pair(d, q), in(0, k));
    }
}
// h_t from h_{t-1}
__device__ __forceinline__ float2 recurrence_next(float2 c, float2 nb, float2 h) {
    return fma_pair(nb, both(-1.f), fma_pair(c, h, h));
}

// The same for the gradients: c[k], and the negated factors of l_t = dL/dh_t in those of x, z and i.
// before(k, h): the state before token k, where h follows from the tokens before it.
template <int n, typename In, typename Before, typename Sum>
__device__ __forceinline__ void recurrence_grads(In&& in, const ChannelRate& r, const GateBound& gb,
                                                 float2 h, Before&& before, float2 (&c)[n],
                                                 float2 (&fx)[n], float2 (&fz)[n], float2 (&fi)[n],
                                                 Sum&& summed) {
    float2 sum;
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const float2 ez = ex2_pair(mul_pair(in(1, k), r.neg_log2));
        const float2 ei = ex2_pair(mul_pair(in(2, k), both(-kLog2e)));
        const float2 sz = rcp1_pair(ez), si = rcp1_pair(ei);
        // 1 - s = e^{-..} s, the exponential limited so that it stays a number where s is zero
        const float2 oz = mul_pair(make_float2(fminf(ez.x, 3e38f), fminf(ez.y, 3e38f)), sz);
        const float2 oi = mul_pair(make_float2(fminf(ei.x, 3e38f), fminf(ei.y, 3e38f)), si);
        sum = k == 0 ? sz : add_pair(sum, sz);
        c[k] = expm1_near(mul_pair(sz, both(gb.scaled)));
        fx[k] = si;
        fz[k] = mul_pair(mul_pair(r.rate_g, sz), oz);
        fi[k] = oi;
    }
    summed(sum);
    for (int j = gb.doublings; j > 0; --j)
#pragma unroll
        for (int k = 0; k < n; ++k) c[k] = twice(c[k]);
#pragma unroll
    for (int k = 0; k < n; ++k) {
        const float2 d = twice(c[k]), q = rsqrt_pair(d);  // -m^2, 1 / m
        const float2 a = add_pair(c[k], both(1.f)), m = mul_pair(d, q);
        const float2 u = mul_pair(fx[k], in(0, k)), mu = mul_pair(m, u);
        fx[k] = mul_pair(m, fx[k]);
        fi[k] = mul_pair(mu, fi[k]);
        // e^A g (1 - s(e^A z)) e^g (e^g / m s(i) x - h)
        h = before(k, h);
        fz[k] = mul_pair(mul_pair(fz[k], a),
                         fma_pair(h, both(-1.f), mul_pair(a, mul_pair(q, u))));
        h = recurrence_next(c[k], mu, h);
    }
}

}  // namespace kda
