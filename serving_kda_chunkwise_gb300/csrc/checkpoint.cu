// checkpoint.cu -- activations kept in 8 bits for the backward pass (declared in include/kda.h).
//
//   e = the smallest exponent in [-127, 121] with max |x| 2^-e < 127.5 over 64 channels of a token
//   code = x 2^-e rounded to the nearest integer (halves to even), in [-127, 127]
// max |x| = f 2^k with f in [1, 2), so e is k - 6 or, when 64 f >= 127.5, k - 5: one comparison of
// bits.  A power of two as scale makes every step exact, so that a value brought back has the bits
// of the formula in bf16 too (a code has 7).
//
// Streaming work: a CTA takes 64 tokens x 256 channels, a lane 8 channels of 8 tokens (all loads
// before any arithmetic), 8 lanes a group.  The tile's exponents meet in shared memory, so that the 64
// of a group are read and written together: byte by byte from the lanes they took as long as the rest.
// Bound by memory: 65,536 x 4096 in bf16 packed in 135 us, 6.0 TB/s, brought back in 120 us, 6.7 TB/s
// (both 355 us where a warp took one group after the other).
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kGroup = 64;
constexpr int kTokens = 64, kChannels = 256;  // of a CTA
constexpr int kEach = kTokens / 8;            // tokens of a warp

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

struct Tile {
    int64_t t0;  // the CTA's first token
    int c0;      // and channel
};
__device__ __forceinline__ Tile tile_of(int D) {
    const unsigned cols = (D + kChannels - 1) / kChannels, t = blockIdx.x / cols;
    return Tile{(int64_t)t * kTokens, (int)(blockIdx.x - t * cols) * kChannels};
}

template <typename IO>
struct Raw;  // 8 values as they are in memory
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16);
            f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    // the largest magnitude's bits as those of an fp32 number, over the 8 lanes of a group (as integers,
    // which puts infinities and then NaN on top)
    __device__ __forceinline__ uint32_t top() const {
        constexpr uint32_t kAbs = 0x7fff7fffu;
        uint32_t m = __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs));
#pragma unroll
        for (int off = 1; off < 8; off <<= 1)
            m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
        return max(m << 16, m & 0xffff0000u);
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
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ uint32_t top() const {
        float f[8];
        get(f);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        return m;
    }
};

template <typename IO>
__global__ void __launch_bounds__(256) pack_kernel(const IO* __restrict__ x, int64_t x_ld,
                                                   int64_t T, int D, int8_t* codes, int8_t* exps) {
    __shared__ int8_t all[kChannels / kGroup][kTokens];
    const Tile tile = tile_of(D);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = tile.c0 + 8 * lane;
    const int64_t t0 = tile.t0 + warp * kEach;
    Raw<IO> raw[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        raw[k].zero();
        if (c < D && t0 + k < T) raw[k].load(x + (t0 + k) * x_ld + c);
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int e = exponent(raw[k].top());
        if ((lane & 7) == 0) all[lane >> 3][warp * kEach + k] = (int8_t)e;
        float v[8];
        raw[k].get(v);
        if (e == 121) {  // the last exponent, under which a code could be 128
            const float most = 127.f * pow2(121);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fminf(fmaxf(v[j], -most), most);
        }
        // v 2^-e + 1.5 2^23 rounds to an integer, halves to even, and has it in its last bits
        const float s = pow2(-e);
        uint32_t out[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float2 r = __ffma2_rn(make_float2(v[4 * j + i], v[4 * j + i + 1]),
                                            make_float2(s, s), make_float2(12582912.f, 12582912.f));
                q[i] = __float_as_uint(r.x);
                q[i + 1] = __float_as_uint(r.y);
            }
            out[j] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
        }
        if (e == -128) out[0] = out[1] = 0u;
        if (c < D && t0 + k < T)
            __stcs(reinterpret_cast<uint2*>(codes + (t0 + k) * D + c), make_uint2(out[0], out[1]));
    }
    __syncthreads();
    const int g = threadIdx.x / kTokens, k = threadIdx.x % kTokens;
    if (tile.c0 + g * kGroup < D && tile.t0 + k < T)
        exps[(int64_t)(tile.c0 / kGroup + g) * T + tile.t0 + k] = all[g][k];
}

template <typename IO>
__global__ void __launch_bounds__(256) unpack_kernel(const int8_t* __restrict__ codes,
                                                     const int8_t* __restrict__ exps, int64_t T,
                                                     int D, IO* x) {
    __shared__ float scale[kChannels / kGroup][kTokens];
    const Tile tile = tile_of(D);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = tile.c0 + 8 * lane;
    const int64_t t0 = tile.t0 + warp * kEach;
    uint2 q[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        q[k] = c < D && t0 + k < T
                   ? __ldcs(reinterpret_cast<const uint2*>(codes + (t0 + k) * D + c))
                   : make_uint2(0u, 0u);
    const int g = threadIdx.x / kTokens, n = threadIdx.x % kTokens;
    if (tile.c0 + g * kGroup < D && tile.t0 + n < T) {
        const int e = exps[(int64_t)(tile.c0 / kGroup + g) * T + tile.t0 + n];
        scale[g][n] = e == -128 ? __int_as_float(0x7fc00000) : pow2(e);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        if (c >= D || t0 + k >= T) continue;
        const float s = scale[lane >> 3][warp * kEach + k];
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)(int8_t)((j < 4 ? q[k].x : q[k].y) >> (8 * (j % 4))) * s;
        store8(x + (t0 + k) * D + c, v);
    }
}

unsigned grid_for(int64_t T, int D) {
    return (unsigned)((T + kTokens - 1) / kTokens * ((D + kChannels - 1) / kChannels));
}

}  // namespace

cudaError_t launch_checkpoint_pack(const void* x, int64_t x_ld, int64_t T, int D, int io_bf16,
                                   int8_t* codes, int8_t* exps, cudaStream_t stream) {
    const unsigned grid = grid_for(T, D);
    ProfScope prof("checkpoint_pack_kernel", stream);
    if (io_bf16)
        pack_kernel<<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(x), x_ld, T, D,
                                              codes, exps);
    else
        pack_kernel<<<grid, 256, 0, stream>>>(static_cast<const float*>(x), x_ld, T, D, codes,
                                              exps);
    return cudaGetLastError();
}

cudaError_t launch_checkpoint_unpack(const int8_t* codes, const int8_t* exps, int64_t T, int D,
                                     int io_bf16, void* x, cudaStream_t stream) {
    const unsigned grid = grid_for(T, D);
    ProfScope prof("checkpoint_unpack_kernel", stream);
    if (io_bf16)
        unpack_kernel<<<grid, 256, 0, stream>>>(codes, exps, T, D, static_cast<__nv_bfloat16*>(x));
    else
        unpack_kernel<<<grid, 256, 0, stream>>>(codes, exps, T, D, static_cast<float*>(x));
    return cudaGetLastError();
}

}  // namespace kda
