// checkpoint.cu -- activations kept in 8 bits for the backward pass (declared in include/kda.h).
//
//   e = the smallest exponent in [-127, 121] with max |x| 2^-e < 127.5 over 64 channels of a token
//   code = x 2^-e rounded to the nearest integer (halves to even), in [-127, 127]
// max |x| = f 2^k with f in [1, 2), so e is k - 6 or, when 64 f >= 127.5, k - 5: one comparison of
// bits.  A power of two as scale makes every step exact, so that a value brought back has the bits
// of the formula in bf16 too (a code has 7).
//
// Streaming work: a lane holds 8 channels, 8 lanes a group.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kGroup = 64;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}

// The exponent for the largest magnitude's bits (sign cleared).
__device__ __forceinline__ int exponent(uint32_t top) {
    if (top >= 0x7f800000u) return -128;
    const int k = (int)(top >> 23) - 127;  // of a denormal number -127, and its e is -127 anyway
    // 64 f >= 127.5 is f >= 1.9921875
    const int e = k - 6 + ((top & 0x7fffffu) >= 0x7f0000u ? 1 : 0);
    return min(max(e, -127), 121);
}

// 2^e for e in [-127, 127], denormal at -127.
__device__ __forceinline__ float pow2(int e) {
    return __int_as_float(e > -127 ? (e + 127) << 23 : 1 << 22);
}

template <typename IO>
__global__ void __launch_bounds__(256) pack_kernel(const IO* __restrict__ x, int64_t x_ld,
                                                   int64_t T, int D, int groups, int8_t* codes,
                                                   int8_t* exps) {
    const int lane = threadIdx.x & 31, sub = lane >> 3;
    // a warp holds four groups of one token
    const int per_row = (groups + 3) / 4;
    const int64_t warps = (int64_t)gridDim.x * 8, items = T * per_row;
    for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < items; w += warps) {
        const int64_t t = w / per_row;
        const int g = (int)(w - t * per_row) * 4 + sub, c = g * kGroup + 8 * (lane & 7);
        const bool live = c < D;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        if (live) load8(x + t * x_ld + c, v);
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
        for (int off = 1; off < 8; off <<= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const int e = exponent(top);
        // by two factors: 2^-e alone leaves fp32's range at both ends
        const float s0 = pow2(-(e >> 1)), s1 = pow2(-(e - (e >> 1)));
        uint32_t out[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = fminf(fmaxf(rintf(v[j] * s0 * s1), -127.f), 127.f);
            out[j / 4] |= ((uint32_t)(int)q & 0xffu) << (8 * (j % 4));
        }
        if (e == -128) out[0] = out[1] = 0u;
        if (live) {
            __stcs(reinterpret_cast<uint2*>(codes + t * D + c), make_uint2(out[0], out[1]));
            if ((lane & 7) == 0) exps[(int64_t)g * T + t] = (int8_t)e;
        }
    }
}

template <typename IO>
__global__ void __launch_bounds__(256) unpack_kernel(const int8_t* __restrict__ codes,
                                                     const int8_t* __restrict__ exps, int64_t T,
                                                     int D, IO* x) {
    const int64_t per_row = D / 8, items = T * per_row;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < items; p += step) {
        const int64_t t = p / per_row;
        const int c = (int)(p - t * per_row) * 8;
        const uint2 q = __ldcs(reinterpret_cast<const uint2*>(codes + t * D + c));
        const int e = exps[(int64_t)(c / kGroup) * T + t];
        const float s = e == -128 ? __int_as_float(0x7fc00000) : pow2(e);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)(int8_t)((j < 4 ? q.x : q.y) >> (8 * (j % 4))) * s;
        store8(x + t * D + c, v);
    }
}

int grid_for(int64_t blocks) {
    const int64_t most = 152 * 16;
    return (int)(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t launch_checkpoint_pack(const void* x, int64_t x_ld, int64_t T, int D, int io_bf16,
                                   int8_t* codes, int8_t* exps, cudaStream_t stream) {
    const int groups = (D + kGroup - 1) / kGroup;
    const int grid = grid_for((T * ((groups + 3) / 4) + 7) / 8);
    ProfScope prof("checkpoint_pack_kernel", stream);
    if (io_bf16)
        pack_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(x), x_ld, T, D,
                                              groups, codes, exps);
    else
        pack_kernel<<<grid, 256, 0, stream>>>(static_cast<const float*>(x), x_ld, T, D, groups,
                                              codes, exps);
    return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const int8_t* codes, const int8_t* exps, int64_t T, int D,
                                     int io_bf16, void* x, cudaStream_t stream) {
    const int grid = grid_for((T * (D / 8) + 255) / 256);
    ProfScope prof("checkpoint_unpack_kernel", stream);
    if (io_bf16)
        unpack_kernel<<<grid, 256, 0, stream>>>(codes, exps, T, D, static_cast<__nv_bfloat16*>(x));
    else
        unpack_kernel<<<grid, 256, 0, stream>>>(codes, exps, T, D, static_cast<float*>(x));
    return cudaGetLastError();
}

}  // namespace kda
