// block_norm.cu -- what stands between a block's output y and the next block's input, and its
// gradients (declared in include/kda.h):
//   n = w_post y / rms(y) (or y),  r' = r + scale s(gate) n,  x' = w_pre r' / rms(r')
// Backward, with f = scale s(gate), G = dL/dr' and hats for values divided by their rms:
//   G  = dr + (w_pre dx - r^ mean(w_pre dx r^)) / rms(r')          (the gradient of r as well)
//   dn = f G,  dy = (w_post dn - y^ mean(w_post dn y^)) / rms(y),  dgate = G f n (1 - s(gate))
//   dscale = sum G s(gate) n,  dw_post = sum dn y^,  dw_pre = sum dx r^
//
// Streaming work: every tensor is read once and written once.  A CTA holds a row at a time, 8 channels
// a thread (16 bytes of bf16), weights and the sums for their gradients in registers.
//   The forward keeps the row in registers, the next one on its way.  Its two means are two sums over
// the CTA one after the other (r' is what the second is of).
//   The gradients read five tensors twice over (before and after the sums): bulk copies bring the next
// rows into shared memory, as many as fit.  Their means are taken together: with q = f w_post y,
//   mean(w_post dn y^) rms(y) D = sum G q = sum dr q + (sum u q - mean(u r^) sum r^ q) / rms(r'),
// u = w_pre dx, so that six sums of one pass give all, and a row costs one barrier.
// All sums are fp32; the only rounding to fewer bits is that of the results.
//   Bound by memory: 32,768 x 4096 in bf16 with gate, scale and both norms 201 us, 6.7 TB/s, the copy
// rate (rows read a second time after the first mean: 1,112 us); gradients with the residual stream in
// fp32 437 us, 6.8 TB/s (plain loads instead of bulk copies 703; six sums by six shuffle reductions
// 532), all in bf16 395 us, 5.4 TB/s, and of rows of 8192 459 us (16,384 rows), 4.7 TB/s: one CTA an SM,
// whose barrier a row no other covers.  With an fp32 residual 298 us (6.3 TB/s), in fp32 227 us (16,384 x
// 4096, 5.9 TB/s): there the 64 registers that 1,024 threads leave spill 4 and 12 bytes.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "tc_util.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kV = 8;          // channels a thread
constexpr int kMaxWarps = 32;  // of a CTA: kMaxBlockNormD / kV threads
constexpr int kWide = 4096;    // the gradients of wider rows take 16 channels a thread
constexpr int kMaxStages = 8;
constexpr int kSmem = 227 * 1024, kStatic = 3 * 1024;  // an SM's shared memory, a CTA's beside its ring

template <typename T>
struct Raw;  // 8 values as they are in memory
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[kV]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16);
            f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[kV]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[kV]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store(float* p, const float (&f)[kV]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
// A thread's values of an fp32 [D] vector, ones where there is none.
__device__ __forceinline__ void weights(const float* w, int c, bool live, float (&f)[kV]) {
#pragma unroll
    for (int e = 0; e < kV; ++e) f[e] = 1.f;
    if (w && live) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(w + c));
        const float4 b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}

// Sums over the CTA's threads, the same in all of them.  buf: alternates from one call to the next, so
// that a call needs one barrier.  (Of six numbers half go to each half of a warp after the first
// step, and the warps' sums are read four at a time by a lane each: 45 instructions, not 170.)
template <int n>
struct Sums {
    static_assert(n == 1 || n == 6, "");
    float part[2][n][kMaxWarps];
};
template <int n>
__device__ __forceinline__ void sum_all(Sums<n>& s, int buf, float (&v)[n]) {
    constexpr unsigned kAll = 0xffffffffu;
    constexpr int kEach = n == 1 ? 1 : n / 2;  // numbers of a half
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    float h[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        if (n == 1) {
            h[k] = v[k] + __shfl_xor_sync(kAll, v[k], 16);
        } else {
            const float keep = lane < 16 ? v[k] : v[n - kEach + k];
            h[k] = keep + __shfl_xor_sync(kAll, lane < 16 ? v[n - kEach + k] : v[k], 16);
        }
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < kEach; ++k) h[k] += __shfl_xor_sync(kAll, h[k], off);
    if (warps == 1) {
#pragma unroll
        for (int k = 0; k < n; ++k) v[k] = __shfl_sync(kAll, h[k % kEach], k / kEach * 16);
        return;
    }
    if (lane % 16 == 0 && (n > 1 || lane == 0))
#pragma unroll
        for (int k = 0; k < kEach; ++k) s.part[buf][lane / 16 * kEach + k][threadIdx.x >> 5] = h[k];
    __syncthreads();
    // four warps' sums of one number a lane (of warps that are not there, zeros)
    constexpr int kLanes = n == 1 ? kMaxWarps / 4 : 4;
    const int k = lane / kLanes;
    float x = 0.f;
    if (k < n) {
        const float4 p = *reinterpret_cast<const float4*>(&s.part[buf][k][lane % kLanes * 4]);
        x = (p.x + p.y) + (p.z + p.w);
    }
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) x += __shfl_xor_sync(kAll, x, off);
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = __shfl_sync(kAll, x, j * kLanes);
}
template <int n>
__device__ __forceinline__ void clear(Sums<n>& s) {
    for (int k = threadIdx.x; k < 2 * n * kMaxWarps; k += blockDim.x)
        (&s.part[0][0][0])[k] = 0.f;
    __syncthreads();
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// s(x), and 1 - s(x) without its cancellation.
struct Gate {
    float s, other;
};
__device__ __forceinline__ Gate gate_of(float x) {
    const float e = exp2_fast(-1.4426950408889634f * x), s = __fdividef(1.f, 1.f + e);
    // (beyond 2^126 the division gives zero, and what is beside it must stay a number)
    return Gate{s, fminf(e, 8e37f) * s};
}

template <typename IO, typename R>
__global__ void __launch_bounds__(1024) norm_kernel(const BlockNormArgs a) {
    __shared__ __align__(16) Sums<1> sums;
    clear(sums);
    const int D = a.D, c = threadIdx.x * kV;
    const bool live = c < D;
    const float over_D = 1.f / D;
    float wn[kV], wx[kV];
    {
        float sc[kV];
        weights(a.w_post, c, live, wn);
        weights(a.scale, c, live, sc);
        weights(a.w_pre, c, live, wx);
#pragma unroll
        for (int e = 0; e < kV; ++e) wn[e] *= sc[e];
    }
    Raw<IO> y, gate;
    Raw<R> r;
    auto fetch = [&](int64_t t) {
        y.zero();
        gate.zero();
        r.zero();
        if (t < a.T && live) {
            y.load(static_cast<const IO*>(a.y) + t * D + c);
            if (a.gate) gate.load(static_cast<const IO*>(a.gate) + t * D + c);
            r.load(static_cast<const R*>(a.r) + t * D + c);
        }
    };
    fetch(blockIdx.x);
    int buf = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float n[kV], h[kV];
        y.get(n);
        float s[1] = {0.f};
        if (a.post_norm) {
#pragma unroll
            for (int e = 0; e < kV; ++e) s[0] = fmaf(n[e], n[e], s[0]);
        }
        if (a.gate) {
            float g[kV];
            gate.get(g);
#pragma unroll
            for (int e = 0; e < kV; ++e) n[e] *= gate_of(g[e]).s;
        }
        r.get(h);
        fetch(t + gridDim.x);
        float inv = 1.f;
        if (a.post_norm) {
            sum_all(sums, buf, s);
            buf ^= 1;
            inv = rsqrtf(s[0] * over_D + a.eps);
        }
        s[0] = 0.f;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            h[e] = fmaf(n[e] * inv, wn[e], h[e]);
            if (live) s[0] = fmaf(h[e], h[e], s[0]);
        }
        sum_all(sums, buf, s);
        buf ^= 1;
        inv = rsqrtf(s[0] * over_D + a.eps);
        if (live) {
#pragma unroll
            for (int e = 0; e < kV; ++e) n[e] = h[e] * inv * wx[e];
            store(static_cast<R*>(a.r_out) + t * D + c, h);
            store(static_cast<IO*>(a.x_out) + t * D + c, n);
        }
    }
}

// Pairs of numbers in one instruction.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

constexpr int kPairs = kV / 2;
__device__ __forceinline__ void read(const __nv_bfloat16* p, float2 (&f)[kPairs]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < kPairs; ++e)
        f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
}
__device__ __forceinline__ void read(const float* p, float2 (&f)[kPairs]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
}
template <typename T>
__device__ __forceinline__ void store(T* p, const float2 (&f)[kPairs]) {
    const float v[kV] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
    store(p, v);
}
__device__ __forceinline__ void weights(const float* w, int c, bool live, float2 (&f)[kPairs]) {
    float v[kV];
    weights(w, c, live, v);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) f[e] = make_float2(v[2 * e], v[2 * e + 1]);
}

// Where a row's tensors are in a stage; those that are not used have no place.
struct Places {
    int y, gate, dx, r, dr, bytes;
};
template <typename IO, typename R>
__host__ __device__ inline Places places(int D, bool y, bool gate, bool dr) {
    Places p{};
    int at = 0;
    auto take = [&](bool used, int elem) {
        const int here = at;
        at += used ? D * elem : 0;
        return here;
    };
    p.y = take(y, sizeof(IO));
    p.gate = take(gate, sizeof(IO));
    p.dx = take(true, sizeof(IO));
    p.r = take(true, sizeof(R));
    p.dr = take(dr, sizeof(R));
    p.bytes = at;
    return p;
}

// kG: groups of 8 channels of a thread, blockDim.x groups apart.  With one, the weights stay in
// registers.
template <typename IO, typename R, int kG>
__global__ void __launch_bounds__(512, 1) norm_bwd_kernel(const __grid_constant__ BlockNormArgs a,
                                                          float* part, int stages, unsigned* err) {
    __shared__ __align__(16) Sums<6> sums;
    __shared__ uint64_t full[kMaxStages];
    extern __shared__ __align__(128) char ring[];
    const int D = a.D;
    const float over_D = 1.f / D;
    // without a norm, gate and scale the block's output is not looked at
    const bool use_y = a.post_norm || a.gate || a.dscale;
    const Places at = places<IO, R>(D, use_y, a.gate, a.dr);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    clear(sums);
    int loads = 0;  // thread 0's
    auto load = [&](int64_t t, int s) {
        if (threadIdx.x != 0 || t >= a.T) return;
        ++loads;
        char* st = ring + s * at.bytes;
        mbar_expect_tx(&full[s], at.bytes);
        const int64_t o = t * D;
        const int io = D * (int)sizeof(IO), re = D * (int)sizeof(R);
        if (use_y) bulk_g2s(st + at.y, static_cast<const IO*>(a.y) + o, io, &full[s]);
        if (a.gate) bulk_g2s(st + at.gate, static_cast<const IO*>(a.gate) + o, io, &full[s]);
        bulk_g2s(st + at.dx, static_cast<const IO*>(a.dx) + o, io, &full[s]);
        bulk_g2s(st + at.r, static_cast<const R*>(a.r) + o, re, &full[s]);
        if (a.dr) bulk_g2s(st + at.dr, static_cast<const R*>(a.dr) + o, re, &full[s]);
    };
    for (int s = 0; s < stages; ++s) load(blockIdx.x + (int64_t)s * gridDim.x, s);

    float2 wn[kPairs], ws[kPairs], wx[kPairs], dwn[kG][kPairs], dws[kG][kPairs], dwx[kG][kPairs];
    auto channel = [&](int g) { return ((int)threadIdx.x + g * (int)blockDim.x) * kV; };
    auto read_weights = [&](int g) {
        const int c = channel(g);
        weights(a.w_post, c, c < D, wn);
        weights(a.scale, c, c < D, ws);
        weights(a.w_pre, c, c < D, wx);
    };
    if (kG == 1) read_weights(0);
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int e = 0; e < kPairs; ++e) dwn[g][e] = dws[g][e] = dwx[g][e] = both(0.f);

    int buf = 0, s = 0, turn = 0;
    bool broken = false;  // (a wait that ran out: the others are not waited for)
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
        const char* st = ring + s * at.bytes;
        const IO* const yp = reinterpret_cast<const IO*>(st + at.y);
        const IO* const gp = reinterpret_cast<const IO*>(st + at.gate);
        const IO* const xp = reinterpret_cast<const IO*>(st + at.dx);
        const R* const rp = reinterpret_cast<const R*>(st + at.r);
        const R* const dp = reinterpret_cast<const R*>(st + at.dr);
        if (!broken) broken = !mbar_wait(&full[s], turn, err);
        float2 v2[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) v2[k] = both(0.f);
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            const int c = channel(g);
            if (c >= D) break;
            if (kG > 1) read_weights(g);
            float2 x[kPairs], r[kPairs];
            read(xp + c, x);
            read(rp + c, r);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                x[e] = mul_pair(x[e], wx[e]);  // u
                v2[1] = fma_pair(r[e], r[e], v2[1]);
                v2[2] = fma_pair(x[e], r[e], v2[2]);
            }
            if (!a.post_norm) continue;
            float2 q[kPairs], d[kPairs];
            read(yp + c, q);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                v2[0] = fma_pair(q[e], q[e], v2[0]);
                q[e] = mul_pair(mul_pair(q[e], wn[e]), ws[e]);
            }
            if (a.gate) {
                read(gp + c, d);
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
                    q[e] = mul_pair(q[e], make_float2(gate_of(d[e].x).s, gate_of(d[e].y).s));
            }
            if (a.dr) {
                read(dp + c, d);
#pragma unroll
                for (int e = 0; e < kPairs; ++e) v2[3] = fma_pair(d[e], q[e], v2[3]);
            }
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                v2[4] = fma_pair(x[e], q[e], v2[4]);
                v2[5] = fma_pair(r[e], q[e], v2[5]);
            }
        }
        float v[6];
#pragma unroll
        for (int k = 0; k < 6; ++k) v[k] = v2[k].x + v2[k].y;
        sum_all(sums, buf, v);
        // (every thread is done with the row before this one: its place is free)
        if (t > blockIdx.x && stages > 1 && !broken)
            load(t + (int64_t)(stages - 1) * gridDim.x, s == 0 ? stages - 1 : s - 1);
        const float inv_y = a.post_norm ? rsqrtf(v[0] * over_D + a.eps) : 1.f;
        const float inv_r = rsqrtf(v[1] * over_D + a.eps);
        // the mean of u r^, and the sum of G q and then the mean of w_post dn y^ from it (each factor next
        // to the sum that it brings to size: a power of inv alone would leave fp32's range)
        const float mean_r = inv_r * over_D * v[2];
        const float mean_y =
            a.post_norm ? inv_y * over_D * (v[3] + inv_r * (v[4] - mean_r * (inv_r * v[5]))) : 0.f;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            const int c = channel(g);
            if (c >= D) break;
            if (kG > 1) read_weights(g);
            const int64_t o = t * D + c;
            float2 G[kPairs], x[kPairs], r[kPairs];
            if (a.dr) {
                read(dp + c, G);
            } else {
#pragma unroll
                for (int e = 0; e < kPairs; ++e) G[e] = both(0.f);
            }
            read(xp + c, x);
            read(rp + c, r);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                const float2 u = mul_pair(x[e], wx[e]), rh = mul_pair(r[e], both(inv_r));
                G[e] = fma_pair(fma_pair(rh, both(-mean_r), u), both(inv_r), G[e]);
                dwx[g][e] = fma_pair(x[e], rh, dwx[g][e]);
            }
            store(static_cast<R*>(a.dr_in) + o, G);
            float2 y[kPairs];
            if (use_y) {
                read(yp + c, y);
            } else {
#pragma unroll
                for (int e = 0; e < kPairs; ++e) y[e] = both(0.f);
            }
            float2 other[kPairs];  // 1 - s(gate)
            if (a.gate) {
                read(gp + c, x);
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    const Gate p = gate_of(x[e].x), q = gate_of(x[e].y);
                    G[e] = mul_pair(G[e], make_float2(p.s, q.s));
                    other[e] = make_float2(p.other, q.other);
                }
            }
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                const float2 yh = mul_pair(y[e], both(inv_y)), n = mul_pair(yh, wn[e]);
                const float2 dn = mul_pair(G[e], ws[e]);
                dws[g][e] = fma_pair(G[e], n, dws[g][e]);
                dwn[g][e] = fma_pair(dn, yh, dwn[g][e]);
                if (a.gate) x[e] = mul_pair(mul_pair(dn, n), other[e]);
                G[e] = a.post_norm
                           ? mul_pair(fma_pair(yh, both(-mean_y), mul_pair(dn, wn[e])), both(inv_y))
                           : dn;
            }
            store(static_cast<IO*>(a.dy) + o, G);
            if (a.gate) store(static_cast<IO*>(a.dgate) + o, x);
        }
        if (stages == 1) {
            __syncthreads();
            if (!broken) load(t + gridDim.x, 0);
        }
        if (++s == stages) {
            s = 0;
            turn ^= 1;
        }
    }
    // a wait that ran out: the copies that are still on their way come first (with a limit), for the
    // shared memory is another kernel's afterwards
    if (threadIdx.x == 0 && broken)
        for (s = 0; s < stages; ++s)
            if (const int fills = ring_fills(loads, s, stages)) mbar_wait(&full[s], fills - 1 & 1, err);
    if (part == nullptr) return;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        const int c = channel(g);
        if (c >= D) break;
        float* out = part + (int64_t)blockIdx.x * 3 * D + c;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            reinterpret_cast<float2*>(out)[e] = dws[g][e];
            reinterpret_cast<float2*>(out + D)[e] = dwn[g][e];
            reinterpret_cast<float2*>(out + 2 * D)[e] = dwx[g][e];
        }
    }
}

// The sums of the blocks' parts in a fixed order: a CTA takes 32 channels of the three vectors, its 32
// warps every 32nd block.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* part, int blocks, int D,
                                                         float* dscale, float* dw_post,
                                                         float* dw_pre) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    grid_dependency_wait();
    float x = 0.f;
    if (c < 3 * D) {
#pragma unroll 4
        for (int b = warp; b < blocks; b += 32) x += part[(int64_t)b * 3 * D + c];
    }
    red[warp][lane] = x;
    __syncthreads();
    if (warp == 0 && c < 3 * D) {
        x = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) x += red[j][lane];
        float* out = c < D ? dscale : c < 2 * D ? dw_post : dw_pre;
        if (out) out[c % D] = x;
    }
}

// For `groups` groups of 8 channels a thread.
int threads_for(int D, int groups = 1) {
    return ((D / kV + groups - 1) / groups + 31) / 32 * 32;
}

// CTAs that fill the GPU, two rows' loads of every thread on their way.
int blocks_for(int64_t T, int threads, int regs_threads) {
    int per_sm = regs_threads / threads;
    if (per_sm > 16) per_sm = 16;
    const int64_t most = 152 * (int64_t)(per_sm < 1 ? 1 : per_sm);
    return (int)(T < most ? T : most);
}

template <typename IO, typename R>
cudaError_t forward(const BlockNormArgs& a) {
    const int threads = threads_for(a.D);
    ProfScope prof("block_norm_kernel", a.stream);
    norm_kernel<IO, R><<<blocks_for(a.T, threads, 1024), threads, 0, a.stream>>>(a);
    return cudaGetLastError();
}

// CTAs of the gradients, 128 registers a thread and 512 threads an SM, and their threads.
int bwd_threads(int D) { return threads_for(D, D > kWide ? 2 : 1); }
int bwd_blocks(int64_t T, int D) { return blocks_for(T, bwd_threads(D), 512); }

template <typename IO, typename R, int kG>
cudaError_t backward_of(const BlockNormArgs& a, float* part, int grid) {
    const int threads = bwd_threads(a.D);
    const Places at = places<IO, R>(a.D, a.post_norm || a.gate || a.dscale, a.gate, a.dr);
    // the rows that an SM's shared memory holds, in equal parts
    const int per_sm = (grid + 151) / 152;
    int stages = (kSmem / per_sm - kStatic) / at.bytes;
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages < 1) return cudaErrorInvalidValue;
    const int smem = stages * at.bytes;
    auto kernel = norm_bwd_kernel<IO, R, kG>;
    // (the same limit whatever the size: another thread may be between this and its launch)
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSmem - kStatic))
        return e;
    ProfScope prof("block_norm_bwd_kernel", a.stream);
    kernel<<<grid, threads, smem, a.stream>>>(a, part, stages, a.dev_err);
    return cudaGetLastError();
}

template <typename IO, typename R>
cudaError_t backward(const BlockNormArgs& a) {
    float* part = a.dscale || a.dw_post || a.dw_pre ? static_cast<float*>(a.workspace) : nullptr;
    const int grid = bwd_blocks(a.T, a.D);
    if (grid > 0) {
        const cudaError_t e = a.D > kWide ? backward_of<IO, R, 2>(a, part, grid)
                                          : backward_of<IO, R, 1>(a, part, grid);
        if (e != cudaSuccess) return e;
    }
    if (part) {
        ProfScope prof("block_norm_sums_kernel", a.stream);
        return launch_dependent(norm_sums_kernel, dim3((3 * a.D + 31) / 32), dim3(1024), 0, a.stream,
                                (const float*)part, grid, a.D, a.dscale, a.dw_post, a.dw_pre);
    }
    return cudaGetLastError();
}

}  // namespace

size_t block_norm_bwd_workspace_size(int D) {
    return (size_t)bwd_blocks((int64_t)1 << 31, D) * 3 * D * sizeof(float);
}

cudaError_t launch_block_norm(const BlockNormArgs& a) {
    if (!a.io_bf16) return forward<float, float>(a);
    return a.r_bf16 ? forward<__nv_bfloat16, __nv_bfloat16>(a) : forward<__nv_bfloat16, float>(a);
}
cudaError_t launch_block_norm_bwd(const BlockNormArgs& a) {
    if (!a.io_bf16) return backward<float, float>(a);
    return a.r_bf16 ? backward<__nv_bfloat16, __nv_bfloat16>(a) : backward<__nv_bfloat16, float>(a);
}

}  // namespace kda
