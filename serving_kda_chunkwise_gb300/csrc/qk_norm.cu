// qk_norm.cu -- RMS norm of every query and key head with the position rotation in the same
// pass, and its gradients (declared in include/kda.h).
//
//   n = w x / sqrt(mean x^2 + eps);   (y_a, y_b) = (n_a cos - n_b sin, n_a sin + n_b cos)
// Backward, with u = the upstream gradient rotated back (the rotation's transpose):
//   dw = sum over rows of u x r,   dx = r (w u) - x r^3 mean(w u x),   r = 1 / sqrt(mean x^2 + eps)
//
// Streaming work: each element is read and written once (backward: x and dy read, dx written).
// A row (one token and head) of d channels is covered by d / 8 lanes with 8 channels each
// (16-byte loads for bf16), so a warp holds 2 (d = 128) or 4 (d = 64) rows at a time and the
// row sums are shuffle reductions.  A warp's task is one token and up to kUnroll row groups of
// that token's heads, so the token's cosines and sines are loaded once a task.  The partner of
// a channel in the (p, p + rot/2) pairing sits in another lane (rot is a multiple of 16, so
// whole lanes pair up) and comes by shuffle; in the interleaved pairing it sits in the same lane.
// All sums and the rotation are fp32; the only rounding to fewer bits is that of the result.
// y may be x: a lane reads its 8 channels before it writes them and no other lane reads them.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;
constexpr int kMaxBwdBlocks = 152 * 4;

template <typename IO>
__device__ __forceinline__ void load8(const IO* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <typename IO>
__device__ __forceinline__ void store8(IO* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}

// What one lane rotates with: its 8 channels' cosines and signed sines (half pairing) or its 4
// pairs' (interleaved, in the first 4 entries).
struct Turn {
    float c[8], s[8];
    int partner;  // lane holding the other members of this lane's pairs (half pairing)
    bool on;      // this lane's channels are rotated
};

template <int D, bool kInter>
__device__ __forceinline__ Turn load_turn(const float* cos_sin, int64_t n_pos,
                                          const int32_t* positions, int rot, int64_t t, int lane,
                                          unsigned* err) {
    constexpr int kLanes = D / 8;
    const int l = lane % kLanes;
    Turn r;
    r.partner = lane;
    r.on = 8 * l < rot;
    if (rot == 0) return r;
    const int64_t p = positions ? (int64_t)__ldg(positions + t) : t;
    if (p < 0 || p >= n_pos) {
        if (lane == 0) atomicOr(err, kDevErrBadPosition);
        r.on = false;
        return r;
    }
    const float* row = cos_sin + p * rot;
    if (kInter) {
        if (r.on) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(row) + l);
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + rot / 2) + l);
            r.c[0] = c.x; r.c[1] = c.y; r.c[2] = c.z; r.c[3] = c.w;
            r.s[0] = s.x; r.s[1] = s.y; r.s[2] = s.z; r.s[3] = s.w;
        }
    } else {
        const int half = rot / 16;  // lanes a half of the rotated channels covers
        const bool second = l >= half;
        if (r.on) {
            r.partner = second ? lane - half : lane + half;
            const int at = second ? l - half : l;
            load8(row + 8 * at, r.c);
            load8(row + rot / 2 + 8 * at, r.s);
            // channel a of a pair takes -sin of its partner, channel b takes +sin
            if (!second)
#pragma unroll
                for (int e = 0; e < 8; ++e) r.s[e] = -r.s[e];
        }
    }
    return r;
}

// Rotates the lane's channels (sign -1: the transposed rotation).  Called by whole warps.
template <bool kInter>
__device__ __forceinline__ void turn(const Turn& r, float sign, int rot, float (&v)[8]) {
    if (rot == 0) return;
    if (kInter) {
        if (r.on)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = v[2 * e], b = v[2 * e + 1], s = sign * r.s[e];
                v[2 * e] = a * r.c[e] - b * s;
                v[2 * e + 1] = a * s + b * r.c[e];
            }
    } else {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, v[e], r.partner);
        if (r.on)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * r.c[e] + o[e] * (sign * r.s[e]);
    }
}

template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = D / 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

struct NormArgs {
    const void *q, *k, *dyq, *dyk;
    int64_t q_ld, k_ld;
    const float *wq, *wk;
    float eps;
    const float* cos_sin;
    int64_t n_pos;
    const int32_t* positions;
    int rot;
    void *q_out, *k_out;  // backward: dq, dk
    float* part;          // backward: [blocks][2][D] partial weight gradients, or nullptr
    int64_t T;
    int Hq, Hk;
    unsigned* err;
};

template <int D, typename IO, bool kInter, bool kBwd>
__global__ void __launch_bounds__(32 * kWarps) norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kLanes = D / 8;
    constexpr int kRows = 32 / kLanes;         // rows a warp holds at a time
    constexpr int kGroup = kRows * kUnroll;    // rows of a task
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % kLanes, sub = lane / kLanes;
    const int nq = (a.Hq + kGroup - 1) / kGroup;
    const int per_token = nq + (a.Hk + kGroup - 1) / kGroup;
    const int64_t tasks = a.T * per_token;
    float dwq[8], dwk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;

    for (int64_t task = (int64_t)blockIdx.x * kWarps + warp; task < tasks;
         task += (int64_t)gridDim.x * kWarps) {
        const int64_t t = task / per_token;
        const int grp = (int)(task - t * per_token);
        const bool is_k = grp >= nq;
        const int H = is_k ? a.Hk : a.Hq;
        const int h0 = (is_k ? grp - nq : grp) * kGroup + sub;
        const IO* x = static_cast<const IO*>(is_k ? a.k : a.q) + t * (is_k ? a.k_ld : a.q_ld) + 8 * l;
        const IO* dy = static_cast<const IO*>(is_k ? a.dyk : a.dyq) + t * H * D + 8 * l;
        IO* y = static_cast<IO*>(is_k ? a.k_out : a.q_out) + t * H * D + 8 * l;
        const float* wp = is_k ? a.wk : a.wq;

        float v[kUnroll][8], u[kBwd ? kUnroll : 1][8];
#pragma unroll
        for (int m = 0; m < kUnroll; ++m) {
            const int h = h0 + m * kRows;
            if (h < H) {
                load8(x + (int64_t)h * D, v[m]);
                if (kBwd) load8(dy + (int64_t)h * D, u[m]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[m][e] = 0.f;
                    if (kBwd) u[m][e] = 0.f;
                }
            }
        }
        const Turn r = load_turn<D, kInter>(a.cos_sin, a.n_pos, a.positions, a.rot, t, lane, a.err);
        float w[8];
        if (wp)
            load8(wp + 8 * l, w);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 1.f;
        float add[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) add[e] = 0.f;
#pragma unroll
        for (int m = 0; m < kUnroll; ++m) {
            const int h = h0 + m * kRows;
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[m][e], v[m][e], ss);
            const float rms = sqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
            const float rinv = 1.f / rms;
            if (!kBwd) {
                float n[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) n[e] = v[m][e] * rinv * w[e];
                turn<kInter>(r, 1.f, a.rot, n);
                if (h < H) store8(y + (int64_t)h * D, n);
            } else {
                turn<kInter>(r, -1.f, a.rot, u[m]);
                float dot = 0.f;
                const bool live = h < H;  // (a dead row with eps = 0 would give 0 * inf)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float hat = v[m][e] * rinv;
                    if (live) add[e] = fmaf(u[m][e], hat, add[e]);
                    u[m][e] *= w[e];
                    dot = fmaf(u[m][e], hat, dot);
                }
                dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[m][e] = rinv * (u[m][e] - v[m][e] * rinv * dot);
                if (live) store8(y + (int64_t)h * D, u[m]);
            }
        }
        if (kBwd) {
            if (is_k)
#pragma unroll
                for (int e = 0; e < 8; ++e) dwk[e] += add[e];
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) dwq[e] += add[e];
        }
    }

    if (kBwd && a.part) {
        __shared__ float red[kWarps][2][D];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = i ? dwk[e] : dwq[e];
#pragma unroll
                for (int off = kLanes; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                if (sub == 0) red[warp][i][8 * l + e] = x;
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {
            float x = 0.f;
#pragma unroll
            for (int j = 0; j < kWarps; ++j) x += red[j][c / D][c % D];
            a.part[(int64_t)blockIdx.x * 2 * D + c] = x;
        }
    }
}

// dw[c] = the sum of the blocks' partials in a fixed order: 1024 / (2 D) threads a channel.
template <int D>
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int blocks, float* dwq,
                                                       float* dwk) {
    constexpr int kParts = 1024 / (2 * D);
    __shared__ float red[kParts][2 * D];
    const int c = threadIdx.x % (2 * D), j = threadIdx.x / (2 * D);
    float x = 0.f;
    for (int b = j; b < blocks; b += kParts) x += part[(int64_t)b * 2 * D + c];
    red[j][c] = x;
    __syncthreads();
    if (j == 0) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) x += red[i][c];
        if (c < D) {
            if (dwq) dwq[c] = x;
        } else if (dwk) {
            dwk[c - D] = x;
        }
    }
}

template <int D, typename IO, bool kBwd>
cudaError_t launch_t(NormArgs a, int interleaved, float* dwq, float* dwk, cudaStream_t s) {
    constexpr int kGroup = 32 / (D / 8) * kUnroll;
    const int64_t per_token = (a.Hq + kGroup - 1) / kGroup + (a.Hk + kGroup - 1) / kGroup;
    const int64_t want = (a.T * per_token + kWarps - 1) / kWarps;
    // the forward runs one task a warp; the backward keeps the weight gradients in registers
    // over a grid-stride loop
    const int64_t cap = kBwd ? (int64_t)kMaxBwdBlocks : ((int64_t)1 << 30);
    const int grid = (int)(want < cap ? want : cap);
    if (grid > 0) {
        ProfScope prof(kBwd ? "qk_norm_bwd_kernel" : "qk_norm_kernel", s);
        if (interleaved)
            norm_kernel<D, IO, true, kBwd><<<grid, 32 * kWarps, 0, s>>>(a);
        else
            norm_kernel<D, IO, false, kBwd><<<grid, 32 * kWarps, 0, s>>>(a);
    }
    if (kBwd && (dwq || dwk)) {
        ProfScope prof("qk_norm_dw_kernel", s);
        norm_dw_kernel<D><<<1, 1024, 0, s>>>(a.part, grid, dwq, dwk);
    }
    return cudaGetLastError();
}

NormArgs to_args(const QkNormArgs& p) {
    NormArgs a{};
    a.q = p.q; a.k = p.k; a.dyq = p.dyq; a.dyk = p.dyk; a.q_ld = p.q_ld; a.k_ld = p.k_ld;
    a.wq = p.wq; a.wk = p.wk; a.eps = p.eps; a.cos_sin = p.cos_sin; a.n_pos = p.n_pos;
    a.positions = p.positions; a.rot = p.rot_dim; a.q_out = p.q_out; a.k_out = p.k_out;
    a.part = (p.dwq || p.dwk) ? static_cast<float*>(p.workspace) : nullptr;
    a.T = p.T; a.Hq = p.Hq; a.Hk = p.Hk; a.err = p.dev_err;
    return a;
}

template <bool kBwd>
cudaError_t dispatch(const QkNormArgs& p) {
    const NormArgs a = to_args(p);
    if (p.d == 128)
        return p.io_bf16 ? launch_t<128, __nv_bfloat16, kBwd>(a, p.interleaved, p.dwq, p.dwk, p.stream)
                         : launch_t<128, float, kBwd>(a, p.interleaved, p.dwq, p.dwk, p.stream);
    return p.io_bf16 ? launch_t<64, __nv_bfloat16, kBwd>(a, p.interleaved, p.dwq, p.dwk, p.stream)
                     : launch_t<64, float, kBwd>(a, p.interleaved, p.dwq, p.dwk, p.stream);
}

}  // namespace

size_t qk_norm_bwd_workspace_size(int d) { return (size_t)kMaxBwdBlocks * 2 * d * sizeof(float); }

cudaError_t launch_qk_norm(const QkNormArgs& p) { return dispatch<false>(p); }
cudaError_t launch_qk_norm_bwd(const QkNormArgs& p) { return dispatch<true>(p); }

}  // namespace kda
