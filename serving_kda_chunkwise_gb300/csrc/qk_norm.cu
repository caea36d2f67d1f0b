// qk_norm.cu -- RMS norm of every query and key head with the position rotation in the same
// pass, and its gradients (declared in include/kda.h).
//
//   n = w x / sqrt(mean x^2 + eps);   (y_a, y_b) = (n_a cos - n_b sin, n_a sin + n_b cos)
// Backward, with u = the upstream gradient rotated back (the rotation's transpose):
//   dw = sum over rows of u x r,   dx = r (w u) - x r^3 mean(w u x),   r = 1 / sqrt(mean x^2 + eps)
//
// Streaming work: each element is read and written once (backward: x and dy read, dx written).
// A row (one token and head) of d channels is covered by d / 8 lanes with two pieces of 4
// channels each, so a warp holds 2 (d = 128) or 4 (d = 64) rows at a time and the row sums are
// shuffle reductions.  The pieces of a lane are 8 neighbouring channels, but in the
// (p, p + rot/2) pairing lanes of rotated channels take channels 4 l .. and rot/2 + 4 l .., so that
// both members of every pair sit in one lane (with whole 16-byte pieces the partner came by 8
// shuffles a row).  A warp's task is one token's queries or keys, some or all of its heads, in
// groups of 1 or 2 times that many rows, the next group's rows on their way while one is worked
// on: the token's position and its row of the table, two dependent loads, are then paid once a
// task.
// Bound by memory and, next, by the instructions (2.5 issued a cycle): 65,536 tokens x 40 heads x
// 128 in bf16 253 us, 1.34 GB at 5.3 TB/s, in fp32 414 us at 6.5.  The gradients by the loads' latency
// (126 registers: a quarter of the warps): 32,768 x 32 heads 184 us, 0.8 GB at 4.4; fp32 289 us at 5.6.
// All sums and the rotation are fp32; the only rounding to fewer bits is that of the result.
// y may be x: a lane reads its 8 channels before it writes them and no other lane reads them.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kWarps = 8;
// Row groups loaded at a time: what keeps some 30 KB a SM on the way within the registers.
template <typename IO>
__host__ __device__ constexpr int unroll(bool bwd) {
    return bwd ? (sizeof(IO) == 2 ? 2 : 1) : (sizeof(IO) == 2 ? 4 : 2);
}
constexpr int kMaxBwdBlocks = 152 * 4;

__device__ __forceinline__ void load4(const float* p, float* v) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}

// Two pieces of 4 channels as they are in memory, loaded ahead of their use.
template <typename IO>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int second) {
        a = __ldcs(reinterpret_cast<const uint2*>(p));
        b = __ldcs(reinterpret_cast<const uint2*>(p + second));
    }
    __device__ __forceinline__ void zero() { a = b = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, int second) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p + second));
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        v[0] = make_float2(a.x, a.y); v[1] = make_float2(a.z, a.w);
        v[2] = make_float2(b.x, b.y); v[3] = make_float2(b.z, b.w);
    }
};

__device__ __forceinline__ void store(__nv_bfloat16* p, int second, const float2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[e].x, v[e].y);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    __stcs(reinterpret_cast<uint2*>(p + second), make_uint2(w[2], w[3]));
}
__device__ __forceinline__ void store(float* p, int second, const float2 (&v)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    __stcs(reinterpret_cast<float4*>(p + second), make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
}

// The cosines and sines of a lane's four pairs.
struct Turn {
    float c[4], s[4];
    bool on;  // the lane's channels are rotated
};

template <int D>
__device__ __forceinline__ Turn load_turn(const float* cos_sin, int64_t n_pos,
                                          const int32_t* positions, int rot, int64_t t, int lane,
                                          unsigned* err) {
    const int l = lane % (D / 8);
    Turn r;
    r.on = 8 * l < rot;
    if (rot == 0) return r;
    const int64_t p = positions ? (int64_t)__ldg(positions + t) : t;
    if (p < 0 || p >= n_pos) {
        if (lane == 0) atomicOr(err, kDevErrBadPosition);
        r.on = false;
        return r;
    }
    if (r.on) {
        load4(cos_sin + p * rot + 4 * l, r.c);
        load4(cos_sin + p * rot + rot / 2 + 4 * l, r.s);
    }
    return r;
}

// Rotates the lane's pairs (the transposed rotation for kBack).
template <bool kInter, bool kBack>
__device__ __forceinline__ void turn(const Turn& r, float2 (&v)[4]) {
    if (!r.on) return;
    if (kInter) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float s = kBack ? -r.s[e] : r.s[e], a = v[e].x, b = v[e].y;
            v[e] = make_float2(a * r.c[e] - b * s, a * s + b * r.c[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 c = make_float2(r.c[2 * e], r.c[2 * e + 1]);
            const float2 s = make_float2(r.s[2 * e], r.s[2 * e + 1]);
            const float2 n = make_float2(-s.x, -s.y), a = v[e], b = v[2 + e];
            v[e] = fma2(b, kBack ? s : n, mul2(a, c));
            v[2 + e] = fma2(a, kBack ? n : s, mul2(b, c));
        }
    }
}

template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = D / 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// The row's sum from the lanes' two pieces.  A lane's pieces are neighbours, or `apart` lanes apart
// (a power of two) where they are split: then each is summed over its neighbours first, which is
// the order in which a row without a rotation is summed, so that its norm has the same bits.
template <int D>
__device__ __forceinline__ float piece_sum(float x, float y, bool split, int apart) {
    if (apart >= D / 8) {  // every lane is split, and to the last step
#pragma unroll
        for (int off = 1; off < D / 8; off <<= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, off);
            y += __shfl_xor_sync(0xffffffffu, y, off);
        }
        return x + y;
    }
    if (!split) {
        x += y;
        y = 0.f;
    }
    if (apart == 0) {
#pragma unroll
        for (int off = 1; off < D / 8; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        return x;
    }
#pragma unroll
    for (int off = 1; off < D / 8; off <<= 1) {
        if (off < apart) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (off == apart) {
            x += y;
            y = 0.f;
        }
        x += __shfl_xor_sync(0xffffffffu, x, off);
    }
    return x + y;
}

struct Side {  // queries or keys
    const void *x, *dy;
    int64_t ld;
    const float* w;
    void* out;     // backward: dx
    int H;
    int parts;     // warps a token's rows are split over
    int64_t warps; // of the launch that work on this side
};

struct NormArgs {
    Side side[2];
    float eps;
    const float* cos_sin;
    int64_t n_pos;
    const int32_t* positions;
    int rot;
    float* part;          // backward: [blocks][2][D] partial weight gradients, or nullptr
    int64_t T;
    unsigned* err;
};

template <int D, typename IO, bool kInter, bool kBwd>
__global__ void __launch_bounds__(32 * kWarps, kBwd ? 2 : 3) norm_kernel(
    const __grid_constant__ NormArgs a) {
    constexpr int kLanes = D / 8;
    constexpr int kRows = 32 / kLanes;         // rows a warp holds at a time
    constexpr int kUnroll = unroll<IO>(kBwd);
    constexpr int kGroup = kRows * kUnroll;    // rows of a group
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % kLanes, sub = lane / kLanes;
    int64_t id = (int64_t)blockIdx.x * kWarps + warp;
    const bool is_k = id >= a.side[0].warps;
    const Side& s = a.side[is_k ? 1 : 0];
    if (is_k) id -= a.side[0].warps;
    const int H = s.H, groups = (H + kGroup - 1) / kGroup;
    const int per_part = (groups + s.parts - 1) / s.parts;
    const int64_t tasks = id < s.warps ? a.T * s.parts : 0;
    // the lane's two pieces of a row
    const bool split = !kInter && 8 * l < a.rot;
    const int first = split ? 4 * l : 8 * l, second = split ? a.rot / 2 : 4;
    // (lanes between a split lane's pieces; other widths sum a lane's pieces first)
    const int wide = kInter ? 0 : a.rot / 8;
    const int apart = (wide & (wide - 1)) == 0 ? wide : 0;
    float2 dw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[e] = make_float2(0.f, 0.f);

    for (int64_t task = id; task < tasks; task += s.warps) {
        const int64_t t = s.parts == 1 ? task : task / s.parts;
        const int g0 = s.parts == 1 ? 0 : (int)(task - t * s.parts) * per_part;
        const int g1 = min(g0 + per_part, groups);
        const IO* xp = static_cast<const IO*>(s.x) + t * s.ld + first;
        const int64_t own = t * H * D + first;
        const IO* up = static_cast<const IO*>(s.dy) + own;
        IO* out = static_cast<IO*>(s.out) + own;

        Raw<IO> x[kUnroll], dy[kBwd ? kUnroll : 1];
        auto fetch = [&](int g) {
#pragma unroll
            for (int m = 0; m < kUnroll; ++m) {
                const int h = g * kGroup + m * kRows + sub;
                x[m].zero();
                if (kBwd) dy[m].zero();
                if (h < H) {
                    x[m].load(xp + h * D, second);
                    if (kBwd) dy[m].load(up + h * D, second);
                }
            }
        };
        if (g0 < g1) fetch(g0);
        const Turn r = load_turn<D>(a.cos_sin, a.n_pos, a.positions, a.rot, t, lane, a.err);
        for (int g = g0; g < g1; ++g) {
            Raw<IO> xc[kUnroll], dc[kBwd ? kUnroll : 1];
#pragma unroll
            for (int m = 0; m < kUnroll; ++m) {
                xc[m] = x[m];
                if (kBwd) dc[m] = dy[m];
            }
            if (g + 1 < g1) fetch(g + 1);
            float w[8];
            if (s.w) {
                load4(s.w + first, w);
                load4(s.w + first + second, w + 4);
            } else
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 1.f;
#pragma unroll
            for (int m = 0; m < kUnroll; ++m) {
                const int h = g * kGroup + m * kRows + sub;
                IO* y = out + h * D;
                float2 v[4];
                xc[m].get(v);
                const float2 q0 = fma2(v[1], v[1], mul2(v[0], v[0]));
                const float2 q1 = fma2(v[3], v[3], mul2(v[2], v[2]));
                const float ss = piece_sum<D>(q0.x + q0.y, q1.x + q1.y, split && apart > 0, apart);
                const float rinv = rsqrtf(ss * (1.f / D) + a.eps);
                const float2 r2 = make_float2(rinv, rinv);
                if (!kBwd) {
                    float2 n[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        n[e] = mul2(mul2(v[e], r2), make_float2(w[2 * e], w[2 * e + 1]));
                    turn<kInter, false>(r, n);
                    if (h < H) store(y, second, n);
                } else {
                    float2 u[4], d2 = make_float2(0.f, 0.f);
                    dc[m].get(u);
                    turn<kInter, true>(r, u);
                    const bool live = h < H;  // (a dead row with eps = 0 would give 0 * inf)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = mul2(v[e], r2);
                        if (live) dw[e] = fma2(u[e], v[e], dw[e]);
                        u[e] = mul2(u[e], make_float2(w[2 * e], w[2 * e + 1]));
                        d2 = fma2(u[e], v[e], d2);
                    }
                    const float dot = -row_sum<D>(d2.x + d2.y) * (1.f / D);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        u[e] = mul2(r2, fma2(v[e], make_float2(dot, dot), u[e]));
                    if (live) store(y, second, u);
                }
            }
        }
    }

    if (kBwd && a.part) {
        __shared__ float red[kWarps][2][D];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x = e & 1 ? dw[e / 2].y : dw[e / 2].x;
#pragma unroll
            for (int off = kLanes; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            if (sub == 0) {
                const int c = first + (e < 4 ? e : second + e - 4);
                red[warp][is_k ? 1 : 0][c] = x;
                red[warp][is_k ? 0 : 1][c] = 0.f;
            }
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

// dw[c] = the sum of the blocks' partials in a fixed order: a CTA takes 32 channels, its 32 warps
// every 32nd block.
template <int D>
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* part, int blocks, float* dwq,
                                                       float* dwk) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float x = 0.f;
#pragma unroll 4
    for (int b = warp; b < blocks; b += 32) x += part[(int64_t)b * 2 * D + c];
    red[warp][lane] = x;
    __syncthreads();
    if (warp == 0) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) x += red[i][lane];
        if (c < D) {
            if (dwq) dwq[c] = x;
        } else if (dwk) {
            dwk[c - D] = x;
        }
    }
}

template <int D, typename IO, bool kBwd>
cudaError_t launch_t(const QkNormArgs& p) {
    constexpr int kGroup = 32 / (D / 8) * unroll<IO>(kBwd);
    NormArgs a{};
    a.side[0] = Side{p.q, p.dyq, p.q_ld, p.wq, p.q_out, p.Hq, 1, 0};
    a.side[1] = Side{p.k, p.dyk, p.k_ld, p.wk, p.k_out, p.Hk, 1, 0};
    a.eps = p.eps; a.cos_sin = p.cos_sin; a.n_pos = p.n_pos; a.positions = p.positions;
    a.rot = p.rot_dim; a.T = p.T; a.err = p.dev_err;
    a.part = (p.dwq || p.dwk) ? static_cast<float*>(p.workspace) : nullptr;
    // A token's rows go to one warp, unless that leaves an SM fewer than some 32 warps.  The forward
    // runs one task a warp; the backward keeps the weight gradients in registers over a
    // grid-stride loop, its warps shared out by the two sides' rows.
    const int64_t fill = 152 * 32;
    const int64_t groups[2] = {(p.Hq + kGroup - 1) / kGroup, (p.Hk + kGroup - 1) / kGroup};
    const int64_t all = groups[0] + groups[1];
    int64_t tasks[2];
    for (int i = 0; i < 2; ++i) {
        const int64_t want = p.T > 0 ? (fill * groups[i] + p.T * all - 1) / (p.T * all) : 1;
        a.side[i].parts = (int)(want < 1 ? 1 : want > groups[i] ? (groups[i] ? groups[i] : 1) : want);
        tasks[i] = groups[i] ? p.T * a.side[i].parts : 0;
        a.side[i].warps = tasks[i];
    }
    if (kBwd && tasks[0] + tasks[1] > (int64_t)kMaxBwdBlocks * kWarps) {
        const int64_t most = (int64_t)kMaxBwdBlocks * kWarps;
        int64_t k = most * groups[1] / all;
        if (groups[1] > 0 && k < 1) k = 1;
        a.side[0].warps = most - k;
        a.side[1].warps = k;
    }
    const int grid = (int)((a.side[0].warps + a.side[1].warps + kWarps - 1) / kWarps);
    if (grid > 0) {
        ProfScope prof(kBwd ? "qk_norm_bwd_kernel" : "qk_norm_kernel", p.stream);
        if (p.interleaved)
            norm_kernel<D, IO, true, kBwd><<<grid, 32 * kWarps, 0, p.stream>>>(a);
        else
            norm_kernel<D, IO, false, kBwd><<<grid, 32 * kWarps, 0, p.stream>>>(a);
    }
    if (kBwd && (p.dwq || p.dwk)) {
        ProfScope prof("qk_norm_dw_kernel", p.stream);
        norm_dw_kernel<D><<<2 * D / 32, 1024, 0, p.stream>>>(a.part, grid, p.dwq, p.dwk);
    }
    return cudaGetLastError();
}

template <bool kBwd>
cudaError_t dispatch(const QkNormArgs& p) {
    if (p.d == 128)
        return p.io_bf16 ? launch_t<128, __nv_bfloat16, kBwd>(p) : launch_t<128, float, kBwd>(p);
    return p.io_bf16 ? launch_t<64, __nv_bfloat16, kBwd>(p) : launch_t<64, float, kBwd>(p);
}

}  // namespace

size_t qk_norm_bwd_workspace_size(int d) { return (size_t)kMaxBwdBlocks * 2 * d * sizeof(float); }

cudaError_t launch_qk_norm(const QkNormArgs& p) { return dispatch<false>(p); }
cudaError_t launch_qk_norm_bwd(const QkNormArgs& p) { return dispatch<true>(p); }

}  // namespace kda
