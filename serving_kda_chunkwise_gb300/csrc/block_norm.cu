// block_norm.cu -- what stands between a block's output y and the next block's input, and its
// gradients (declared in include/kda.h):
//   n = w_post y / rms(y) (or y),  r' = r + scale s(gate) n,  x' = w_pre r' / rms(r')
// Backward, with f = scale s(gate), G = dL/dr' and hats for values divided by their rms:
//   G  = dr + (w_pre dx - r^ mean(w_pre dx r^)) / rms(r')          (the gradient of r as well)
//   dn = f G,  dy = (w_post dn - y^ mean(w_post dn y^)) / rms(y),  dgate = G f n (1 - s(gate))
//   dscale = sum G s(gate) n,  dw_post = sum dn y^,  dw_pre = sum dx r^
//
// Streaming work: every tensor is read once and written once.  A CTA holds a row at a time in
// registers, 8 channels a thread (16 bytes of bf16), and goes over its rows with the next one on its
// way; weights, and the sums for their gradients, stay in registers.  The forward's two means are
// two sums over the CTA one after the other (r' is what the second is of).  The gradients' are taken
// together: with q = f w_post y,
//   mean(w_post dn y^) rms(y) D = sum G q = sum dr q + (sum u q - mean(u r^) sum r^ q) / rms(r'),
// u = w_pre dx, so that six sums of one pass give all, and a row costs one barrier.
// All sums are fp32; the only rounding to fewer bits is that of the results.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kV = 8;          // channels a thread
constexpr int kMaxWarps = 32;  // of a CTA: kMaxBlockNormD / kV threads
constexpr int kMaxBlocks = 152 * 8;
// rows wider than this keep the gradients' sums in shared memory: 1,024 threads have no registers
constexpr int kWide = 4096;

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
// that a call needs one barrier.
template <int n>
struct Sums {
    float part[2][n][kMaxWarps];
};
template <int n>
__device__ __forceinline__ void sum_all(Sums<n>& s, int buf, float (&v)[n]) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < n; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    const int warps = blockDim.x / 32;
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < n; ++k) s.part[buf][k][threadIdx.x >> 5] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] = 0.f;
    for (int w = 0; w < warps; w += 4)  // (the unused ones are zeros)
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float4 p = *reinterpret_cast<const float4*>(&s.part[buf][k][w]);
            v[k] += (p.x + p.y) + (p.z + p.w);
        }
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

// kWideRows: rows of more than kWide channels, whose sums are kept in shared memory ([3][D]).
template <typename IO, typename R, bool kWideRows>
__global__ void __launch_bounds__(kWideRows ? 1024 : 512, 1) norm_bwd_kernel(const BlockNormArgs a,
                                                                            float* part) {
    __shared__ __align__(16) Sums<6> sums;
    extern __shared__ __align__(16) float kept[];
    clear(sums);
    const int D = a.D, c = threadIdx.x * kV;
    const bool live = c < D;
    const float over_D = 1.f / D;
    // without a norm, gate and scale the block's output is not looked at
    const bool use_y = a.post_norm || a.gate || a.dscale;
    float wn[kV], ws[kV], wx[kV], dwn[kV], dws[kV], dwx[kV];
    auto read_weights = [&] {
        weights(a.w_post, c, live, wn);
        weights(a.scale, c, live, ws);
        weights(a.w_pre, c, live, wx);
    };
    if (!kWideRows) read_weights();
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        dwn[e] = dws[e] = dwx[e] = 0.f;
        if (kWideRows && live) kept[c + e] = kept[D + c + e] = kept[2 * D + c + e] = 0.f;
    }
    Raw<IO> yr, gr, xr;
    Raw<R> rr, dr;
    auto fetch = [&](int64_t t) {
        yr.zero();
        gr.zero();
        xr.zero();
        rr.zero();
        dr.zero();
        if (t < a.T && live) {
            const int64_t at = t * D + c;
            if (use_y) yr.load(static_cast<const IO*>(a.y) + at);
            if (a.gate) gr.load(static_cast<const IO*>(a.gate) + at);
            xr.load(static_cast<const IO*>(a.dx) + at);
            rr.load(static_cast<const R*>(a.r) + at);
            if (a.dr) dr.load(static_cast<const R*>(a.dr) + at);
        }
    };
    fetch(blockIdx.x);
    int buf = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
        const Raw<IO> y_ = yr, g_ = gr, x_ = xr;
        const Raw<R> r_ = rr, d_ = dr;
        fetch(t + gridDim.x);
        float v[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (kWideRows) read_weights();
        {
            float y[kV], g[kV], x[kV], r[kV], d[kV];
            y_.get(y);
            g_.get(g);
            x_.get(x);
            r_.get(r);
            d_.get(d);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float u = x[e] * wx[e];
                v[1] = fmaf(r[e], r[e], v[1]);
                v[2] = fmaf(u, r[e], v[2]);
                if (a.post_norm) {
                    const float q = y[e] * wn[e] * ws[e] * (a.gate ? gate_of(g[e]).s : 1.f);
                    v[0] = fmaf(y[e], y[e], v[0]);
                    v[3] = fmaf(d[e], q, v[3]);
                    v[4] = fmaf(u, q, v[4]);
                    v[5] = fmaf(r[e], q, v[5]);
                }
            }
        }
        sum_all(sums, buf, v);
        const float inv_y = a.post_norm ? rsqrtf(v[0] * over_D + a.eps) : 1.f;
        const float inv_r = rsqrtf(v[1] * over_D + a.eps);
        // G = dr + inv_r u - back r
        const float back = inv_r * inv_r * inv_r * (v[2] * over_D);
        const float dot = a.post_norm ? inv_y * inv_y * over_D * (v[3] + inv_r * v[4] - back * v[5]) : 0.f;
        if (!live) continue;
        if (kWideRows) {
            asm volatile("" ::: "memory");  // (read again, not kept)
            read_weights();
        }
        float y[kV], x[kV], r[kV], G[kV];
        y_.get(y);
        x_.get(x);
        r_.get(r);
        d_.get(G);
#pragma unroll
        for (int e = 0; e < kV; ++e) G[e] = fmaf(-back, r[e], fmaf(inv_r, x[e] * wx[e], G[e]));
        const int64_t at = t * D + c;
        store(static_cast<R*>(a.dr_in) + at, G);
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            r[e] = x[e] * r[e] * inv_r;  // dw_pre's
            dwx[e] += r[e];
        }
        float g[kV], dy[kV];
        g_.get(g);
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            const Gate s = a.gate ? gate_of(g[e]) : Gate{1.f, 0.f};
            const float yh = y[e] * inv_y, gs = G[e] * s.s, dn = gs * ws[e];
            dy[e] = inv_y * (dn * wn[e]) - y[e] * (inv_y * dot);
            if (!a.post_norm) dy[e] = dn;
            g[e] = dn * yh * wn[e] * s.other;
            x[e] = gs * yh * wn[e];  // dscale's
            y[e] = dn * yh;          // dw_post's
            dws[e] += x[e];
            dwn[e] += y[e];
        }
        store(static_cast<IO*>(a.dy) + at, dy);
        if (a.gate) store(static_cast<IO*>(a.dgate) + at, g);
        if (kWideRows) {
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                kept[c + e] += x[e];
                kept[D + c + e] += y[e];
                kept[2 * D + c + e] += r[e];
            }
        }
    }
    if (part && live) {
        float* out = part + (int64_t)blockIdx.x * 3 * D + c;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            out[e] = kWideRows ? kept[c + e] : dws[e];
            out[D + e] = kWideRows ? kept[D + c + e] : dwn[e];
            out[2 * D + e] = kWideRows ? kept[2 * D + c + e] : dwx[e];
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

int threads_for(int D) { return (D / kV + 31) / 32 * 32; }

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

template <typename IO, typename R>
cudaError_t backward(const BlockNormArgs& a) {
    float* part = a.dscale || a.dw_post || a.dw_pre ? static_cast<float*>(a.workspace) : nullptr;
    const int threads = threads_for(a.D);
    int grid = blocks_for(a.T, threads, 512);
    if (grid > kMaxBlocks) grid = kMaxBlocks;
    if (grid > 0) {
        ProfScope prof("block_norm_bwd_kernel", a.stream);
        if (a.D > kWide) {
            const int smem = 3 * a.D * (int)sizeof(float);
            if (cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<IO, R, true>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
                return e;
            norm_bwd_kernel<IO, R, true><<<grid, threads, smem, a.stream>>>(a, part);
        } else {
            norm_bwd_kernel<IO, R, false><<<grid, threads, 0, a.stream>>>(a, part);
        }
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
    return (size_t)blocks_for(kMaxBlocks, threads_for(D), 512) * 3 * D * sizeof(float);
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
