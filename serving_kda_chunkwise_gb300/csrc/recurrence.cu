// recurrence.cu -- the gated recurrence of single channels (declared in include/kda.h): packed
// forward, gradients (from whole or 8-bit inputs) and the single-token step.
//
// One thread a sequence and channel, token by token; the gradients go back in pieces of 64 tokens,
// whose states are formed again from the state at the piece's start (the edges).
#include "kda_internal.h"
#include "recurrence_math.cuh"

namespace kda {
namespace {

constexpr int kEdge = 64;   // tokens from one edge to the next
constexpr int kGroup = 64;  // channels that share an exponent of packed inputs

template <typename In>
__device__ __forceinline__ float input(const void* p, int64_t ld, const int8_t*, int64_t, int64_t t,
                                       int c) {
    return to_f32(static_cast<const In*>(p)[t * ld + c]);
}
template <>
__device__ __forceinline__ float input<int8_t>(const void* p, int64_t ld, const int8_t* exps,
                                               int64_t T, int64_t t, int c) {
    const int e = exps[(int64_t)(c / kGroup) * T + t];
    if (e == -128) return __int_as_float(0x7fc00000);
    return ldexpf((float)static_cast<const int8_t*>(p)[t * ld + c], e);
}

template <typename In>
__device__ __forceinline__ void inputs(const RecurrenceArgs& a, int64_t t, int c, float& x,
                                       float& z, float& i) {
    x = input<In>(a.x, a.x_ld, a.x_exps, a.T_total, t, c);
    z = input<In>(a.z, a.z_ld, a.z_exps, a.T_total, t, c);
    i = input<In>(a.i, a.i_ld, a.i_exps, a.T_total, t, c);
}

template <typename In, typename IO>
__global__ void __launch_bounds__(128) forward_kernel(const RecurrenceArgs a) {
    const int c = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y;
    if (c >= a.D) return;
    int64_t b, e;
    seq_range(a.cu_seqlens, n, a.N, a.T_total, a.dev_err, b, e);
    float h = a.h0 ? a.h0[(int64_t)n * a.D + c] : 0.f;
    if (b < e) {
        const ChannelRate r = channel_rate(a.A_log[c]);
        for (int64_t t = b; t < e; ++t) {
            if (a.edges && t % kEdge == 0) a.edges[t / kEdge * a.D + c] = h;
            float x, z, i;
            inputs<In>(a, t, c, x, z, i);
            const Step s = recurrence_step(x, z, i, r.neg_log2, a.g_min);
            h = recurrence_next(s.c, s.b, h);
            if (a.y) static_cast<IO*>(a.y)[t * a.D + c] = from_f32<IO>(h);
        }
    }
    if (a.h_out) a.h_out[(int64_t)n * a.D + c] = h;
}

template <typename In, typename IO>
__global__ void __launch_bounds__(128) backward_kernel(const RecurrenceArgs a, float* part) {
    const int c = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y;
    if (c >= a.D) return;
    int64_t b, e;
    seq_range(a.cu_seqlens, n, a.N, a.T_total, a.dev_err, b, e);
    float l = a.dh_out ? a.dh_out[(int64_t)n * a.D + c] : 0.f, dA = 0.f;
    if (b < e) {
        const ChannelRate r = channel_rate(a.A_log[c]);
        float before[kEdge];
        for (int64_t end = e; end > b;) {
            const int64_t edge = (end - 1) / kEdge * kEdge, from = edge < b ? b : edge;
            float h = edge < b ? (a.h0 ? a.h0[(int64_t)n * a.D + c] : 0.f)
                               : a.edges[edge / kEdge * a.D + c];
            for (int64_t t = from; t < end; ++t) {
                float x, z, i;
                inputs<In>(a, t, c, x, z, i);
                before[t - from] = h;
                const Step s = recurrence_step(x, z, i, r.neg_log2, a.g_min);
                h = recurrence_next(s.c, s.b, h);
            }
            for (int64_t t = end - 1; t >= from; --t) {
                float x, z, i;
                inputs<In>(a, t, c, x, z, i);
                l += to_f32(static_cast<const IO*>(a.dy)[t * a.dy_ld + c]);
                const StepGrad s =
                    recurrence_grad(x, z, i, r.rate, r.neg_log2, a.g_min, before[t - from]);
                const float dz = l * s.dz;
                static_cast<IO*>(a.dx)[t * a.D + c] = from_f32<IO>(l * s.dx);
                static_cast<IO*>(a.di)[t * a.D + c] = from_f32<IO>(l * s.di);
                static_cast<IO*>(a.dz)[t * a.D + c] = from_f32<IO>(dz);
                // (an infinite z has a gradient of zero)
                dA += dz == 0.f ? 0.f : dz * z;
                l = recurrence_next(recurrence_step(x, z, i, r.neg_log2, a.g_min).c, 0.f, l);
            }
            end = from;
        }
    }
    if (a.dh0) a.dh0[(int64_t)n * a.D + c] = l;
    if (a.dA_log) part[(int64_t)n * a.D + c] = dA;
}

// dA_log[c] = the sum of the sequences' parts in order.
__global__ void __launch_bounds__(128) rate_kernel(const float* part, int N, int D, float* dA) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= D) return;
    float x = 0.f;
    for (int n = 0; n < N; ++n) x += part[(int64_t)n * D + c];
    dA[c] = x;
}

template <typename IO>
__global__ void __launch_bounds__(128) step_kernel(const IO* x, int64_t x_ld, const IO* z,
                                                   int64_t z_ld, const IO* i, int64_t i_ld,
                                                   const float* A_log, float g_min, float* h,
                                                   const int32_t* slots, int n_slots, int D, IO* y,
                                                   unsigned* err) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    const int64_t n = blockIdx.y;
    if (c >= D) return;
    int64_t slot = slots ? slots[n] : n;
    if (slot >= n_slots) {
        atomicOr(err, kDevErrBadSlot);
        slot = -1;
    }
    float v = 0.f;
    if (slot >= 0) {
        const Step s = recurrence_step(to_f32(x[n * x_ld + c]), to_f32(z[n * z_ld + c]),
                                       to_f32(i[n * i_ld + c]), channel_rate(A_log[c]).neg_log2,
                                       g_min);
        v = recurrence_next(s.c, s.b, h[slot * D + c]);
        h[slot * D + c] = v;
    }
    y[n * D + c] = from_f32<IO>(v);
}

size_t edges_bytes(int64_t T, int D) {
    return ((size_t)((T + kEdge - 1) / kEdge) * D * sizeof(float) + 255) / 256 * 256;
}

template <typename In, typename IO>
cudaError_t forward(const RecurrenceArgs& a) {
    const dim3 grid((a.D + 127) / 128, a.N);
    ProfScope prof("recurrence_kernel", a.stream);
    forward_kernel<In, IO><<<grid, 128, 0, a.stream>>>(a);
    return cudaGetLastError();
}

template <typename In, typename IO>
cudaError_t backward(RecurrenceArgs a) {
    float* part = static_cast<float*>(a.workspace);
    if (a.edges == nullptr) {
        RecurrenceArgs f = a;
        f.edges = a.edges = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                                     ((size_t)a.N * a.D * 4 + 255) / 256 * 256);
        f.y = nullptr;
        f.h_out = nullptr;
        if (cudaError_t e = forward<In, IO>(f)) return e;
    }
    const dim3 grid((a.D + 127) / 128, a.N);
    {
        ProfScope prof("recurrence_bwd_kernel", a.stream);
        backward_kernel<In, IO><<<grid, 128, 0, a.stream>>>(a, part);
    }
    if (a.dA_log) {
        ProfScope prof("recurrence_rate_kernel", a.stream);
        rate_kernel<<<grid.x, 128, 0, a.stream>>>(part, a.N, a.D, a.dA_log);
    }
    return cudaGetLastError();
}

}  // namespace

size_t recurrence_fwd_workspace_size(int64_t, int, int) { return 0; }
size_t recurrence_bwd_workspace_size(int64_t T, int N, int D) {
    return ((size_t)N * D * 4 + 255) / 256 * 256 + edges_bytes(T, D);
}

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a) {
    return a.io_bf16 ? forward<__nv_bfloat16, __nv_bfloat16>(a) : forward<float, float>(a);
}
cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a) {
    if (a.packed)
        return a.io_bf16 ? backward<int8_t, __nv_bfloat16>(a) : backward<int8_t, float>(a);
    return a.io_bf16 ? backward<__nv_bfloat16, __nv_bfloat16>(a) : backward<float, float>(a);
}

cudaError_t launch_recurrence_step(const void* x, int64_t x_ld, const void* z, int64_t z_ld,
                                   const void* i, int64_t i_ld, const float* A_log, float g_min,
                                   float* h, const int32_t* slots, int n_slots, int N, int D,
                                   int io_bf16, void* y, unsigned* dev_err, cudaStream_t stream) {
    const dim3 grid((D + 127) / 128, N);
    ProfScope prof("recurrence_step_kernel", stream);
    if (io_bf16) {
        using T = __nv_bfloat16;
        step_kernel<T><<<grid, 128, 0, stream>>>(
            static_cast<const T*>(x), x_ld, static_cast<const T*>(z), z_ld,
            static_cast<const T*>(i), i_ld, A_log, g_min, h, slots, n_slots, D,
            static_cast<T*>(y), dev_err);
    } else {
        step_kernel<float><<<grid, 128, 0, stream>>>(
            static_cast<const float*>(x), x_ld, static_cast<const float*>(z), z_ld,
            static_cast<const float*>(i), i_ld, A_log, g_min, h, slots, n_slots, D,
            static_cast<float*>(y), dev_err);
    }
    return cudaGetLastError();
}

}  // namespace kda
