// block_norm.cu -- what stands between a block's output y and the next block's input, and its
// gradients (declared in include/kda.h):
//   n = w_post y / rms(y) (or y),  r' = r + scale s(gate) n,  x' = w_pre r' / rms(r')
// Backward, with f = scale s(gate), G = dL/dr' and hats for values divided by their rms:
//   G  = dr + (w_pre dx - r^ mean(w_pre dx r^)) / rms(r')          (the gradient of r as well)
//   dn = f G,  dy = (w_post dn - y^ mean(w_post dn y^)) / rms(y),  dgate = G f n (1 - s(gate))
//   dscale = sum G s(gate) n,  dw_post = sum dn y^,  dw_pre = sum dx r^
//
// One CTA a row, which it keeps in shared memory.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kBwdBlocks = 152;

__device__ __forceinline__ float logistic(float x) { return 1.f / (1.f + expf(-x)); }

__device__ __forceinline__ float block_sum(float x) {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x += part[w];
    return x;
}

template <typename IO, typename R>
__global__ void __launch_bounds__(kThreads) norm_kernel(const BlockNormArgs a) {
    extern __shared__ float row[];
    const int D = a.D;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const IO* y = static_cast<const IO*>(a.y) + t * D;
        const IO* gate = a.gate ? static_cast<const IO*>(a.gate) + t * D : nullptr;
        const R* r = static_cast<const R*>(a.r) + t * D;
        float s = 0.f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float v = to_f32(y[c]);
            s = fmaf(v, v, s);
        }
        const float inv = a.post_norm ? rsqrtf(block_sum(s) / D + a.eps) : 1.f;
        s = 0.f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            float n = to_f32(y[c]) * inv;
            if (a.w_post) n *= a.w_post[c];
            if (a.scale) n *= a.scale[c];
            if (gate) n *= logistic(to_f32(gate[c]));
            n += to_f32(r[c]);
            row[c] = n;
            s = fmaf(n, n, s);
        }
        const float inv2 = rsqrtf(block_sum(s) / D + a.eps);
        for (int c = threadIdx.x; c < D; c += kThreads) {
            static_cast<R*>(a.r_out)[t * D + c] = from_f32<R>(row[c]);
            static_cast<IO*>(a.x_out)[t * D + c] =
                from_f32<IO>(row[c] * inv2 * (a.w_pre ? a.w_pre[c] : 1.f));
        }
    }
}

template <typename IO, typename R>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const BlockNormArgs a, float* part) {
    extern __shared__ float row[];  // G of the row
    const int D = a.D;
    float* sums = part ? part + (int64_t)blockIdx.x * 3 * D : nullptr;
    if (sums)
        for (int c = threadIdx.x; c < 3 * D; c += kThreads) sums[c] = 0.f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const IO* y = static_cast<const IO*>(a.y) + t * D;
        const IO* dx = static_cast<const IO*>(a.dx) + t * D;
        const IO* gate = a.gate ? static_cast<const IO*>(a.gate) + t * D : nullptr;
        const R* r = static_cast<const R*>(a.r) + t * D;
        const R* dr = a.dr ? static_cast<const R*>(a.dr) + t * D : nullptr;
        float sy = 0.f, sr = 0.f, sx = 0.f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float v = to_f32(y[c]), w = to_f32(r[c]);
            sy = fmaf(v, v, sy);
            sr = fmaf(w, w, sr);
            sx = fmaf(to_f32(dx[c]) * (a.w_pre ? a.w_pre[c] : 1.f), w, sx);
        }
        const float inv_y = a.post_norm ? rsqrtf(block_sum(sy) / D + a.eps) : 1.f;
        const float inv_r = rsqrtf(block_sum(sr) / D + a.eps);
        const float dot_r = block_sum(sx) * inv_r / D;
        float sd = 0.f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float u = to_f32(dx[c]) * (a.w_pre ? a.w_pre[c] : 1.f);
            const float G = (dr ? to_f32(dr[c]) : 0.f) + inv_r * (u - to_f32(r[c]) * inv_r * dot_r);
            row[c] = G;
            float dn = G;
            if (gate) dn *= logistic(to_f32(gate[c]));
            if (a.scale) dn *= a.scale[c];
            if (a.w_post) dn *= a.w_post[c];
            sd = fmaf(dn, to_f32(y[c]), sd);
        }
        const float dot_y = a.post_norm ? block_sum(sd) * inv_y / D : 0.f;
        for (int c = threadIdx.x; c < D; c += kThreads) {
            const float G = row[c], yh = to_f32(y[c]) * inv_y;
            const float sg = gate ? logistic(to_f32(gate[c])) : 1.f;
            const float sc = a.scale ? a.scale[c] : 1.f, w = a.w_post ? a.w_post[c] : 1.f;
            static_cast<R*>(a.dr_in)[t * D + c] = from_f32<R>(G);
            const float dn = G * sg * sc;
            const float dy = a.post_norm ? inv_y * (dn * w - yh * dot_y) : dn;
            static_cast<IO*>(a.dy)[t * D + c] = from_f32<IO>(dy);
            if (gate) {
                // 1 - s(gate) without its cancellation
                const float os = logistic(-to_f32(gate[c]));
                static_cast<IO*>(a.dgate)[t * D + c] = from_f32<IO>(dn * yh * w * os);
            }
            if (sums) {
                sums[c] += G * sg * yh * w;
                sums[D + c] += dn * yh;
                sums[2 * D + c] += to_f32(dx[c]) * to_f32(r[c]) * inv_r;
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads) norm_sums_kernel(const float* part, int blocks, int D,
                                                             float* dscale, float* dw_post,
                                                             float* dw_pre) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= 3 * D) return;
    float x = 0.f;
    for (int b = 0; b < blocks; ++b) x += part[(int64_t)b * 3 * D + c];
    float* out = c < D ? dscale : c < 2 * D ? dw_post : dw_pre;
    if (out) out[c % D] = x;
}

template <typename IO, typename R>
cudaError_t forward(const BlockNormArgs& a) {
    const int grid = (int)(a.T < 152 * 8 ? a.T : 152 * 8);
    ProfScope prof("block_norm_kernel", a.stream);
    norm_kernel<IO, R><<<grid, kThreads, a.D * sizeof(float), a.stream>>>(a);
    return cudaGetLastError();
}

template <typename IO, typename R>
cudaError_t backward(const BlockNormArgs& a) {
    float* part = a.dscale || a.dw_post || a.dw_pre ? static_cast<float*>(a.workspace) : nullptr;
    const int grid = (int)(a.T < kBwdBlocks ? a.T : kBwdBlocks);
    if (grid > 0) {
        ProfScope prof("block_norm_bwd_kernel", a.stream);
        norm_bwd_kernel<IO, R><<<grid, kThreads, a.D * sizeof(float), a.stream>>>(a, part);
    }
    if (part) {
        ProfScope prof("block_norm_sums_kernel", a.stream);
        norm_sums_kernel<<<(3 * a.D + kThreads - 1) / kThreads, kThreads, 0, a.stream>>>(
            part, grid, a.D, a.dscale, a.dw_post, a.dw_pre);
    }
    return cudaGetLastError();
}

}  // namespace

size_t block_norm_bwd_workspace_size(int D) { return (size_t)kBwdBlocks * 3 * D * sizeof(float); }

cudaError_t launch_block_norm(const BlockNormArgs& a) {
    if (!a.io_bf16) return forward<float, float>(a);
    return a.r_bf16 ? forward<__nv_bfloat16, __nv_bfloat16>(a) : forward<__nv_bfloat16, float>(a);
}
cudaError_t launch_block_norm_bwd(const BlockNormArgs& a) {
    if (!a.io_bf16) return backward<float, float>(a);
    return a.r_bf16 ? backward<__nv_bfloat16, __nv_bfloat16>(a) : backward<__nv_bfloat16, float>(a);
}

}  // namespace kda
