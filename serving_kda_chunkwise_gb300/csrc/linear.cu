// linear.cu -- linear attention with one decay per head (declared in include/kda.h):
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t
// its gradients and its single-token step.  linear_common.cuh says how the forward and the
// three gradients are instances of one call and how sequences are cut into segments.
//
// Launches of a call over sequences longer than a segment:
//   1. (bf16) decays: what the chunks' products need of the log decays, see linear_tc.cu;
//   2. segment sums: each segment's own contribution to the state, and its summed log decay; for
//      bf16 also the states after sequences of one segment;
//   3. edges: the state at every segment's edge (a scan over a sequence's segments) and, for bf16,
//      after the sequence;
//   4. outputs: every segment from its edge state (fp32: and the states after the sequences);
//   5. (gradients) the decays'.
// When no sequence can be longer than a segment, 3 falls away, and 2 where no state is wanted.
// With S_out in S0's place the states of bf16 sequences of one segment come last, for the outputs
// read S0. Each launch but the first is a programmatic dependent of the one before: it is set up
// beside it and waits before it reads what that wrote (every kernel waits, so that a launch's end
// is that of all before it).
//
// The gradient of g:  dg_t = sum_{s >= t} (q_s . dq_s - k_s . dk_s) + <S_T, dS_out>.  Both dot
// products hold the token's own term (q_s . k_s) (v_s . do_s), the only one without a decay.  It is
// left out of both: carried along, its rounding would drown the rest where decays are strong (dg of
// a head is of the size of e^g; at g = -10 everywhere it came out 1 % off, a fixed decay's 100
// times too large).  Taken over a long sequence the sum would gather the rounding of every later
// token. At every segment's edges it is <S, D>, from states that are at hand, so the sums run
// inside a segment, from the anchor at its start: dg_t = <S, D> - sum_{s < t} (...).  What they
// miss the anchor at its end by is their rounding, and is taken back token by token in proportion
// to the squares of the terms' sizes, as independent errors are best shared out.  (From the end
// they would begin, at a sequence's last token, with <S_T, dS_out>, in which that token's own k v^T
// has no decay either.)
#include <algorithm>
#include <cstdlib>
#include <cstring>

#include "linear_common.cuh"
#include "linear_tc.h"

namespace kda {
namespace {

using lin::Call;
using lin::Calls;
using lin::Problem;
using lin::Segment;

// -------------------------------------------------- token by token, CUDA cores --
// A CTA of 128 threads holds a da x 64 block of the state in registers (a lane two columns, a warp
// a quarter of the rows, in pairs) and walks the segment's tokens, 16 at a time through shared
// memory, the next 16 on their way in registers meanwhile.  fp32 throughout, so that fp32 inputs
// keep fp32 accuracy.  The state decays by S += S (e^g - 1) unless g is far below 0: e^g itself
// rounds near 1, and one decay for all tokens would round the same way at every one of them. Bound
// by its three (sums: two) fp32 operations per state element and token: at 65,536 tokens x 16 heads
// x 128 the outputs take 2,163 us, 64 % of the fp32 rate, the sums 1,207 us, 77 %, the three of the
// gradients 7,543 us; at 2,048 + 1,531 tokens x 8 heads, 64 x 128, 45, 30 and 143 us (with one
// column a lane and no tile on its way outputs and sums took 98 and 69 us).
constexpr int kCols = 64;
constexpr int kDotCols = 32;
constexpr int kTile = 16;
constexpr float kNear = -0.5f;  // below it e^g - 1 has no more bits of e^g than e^g itself

template <typename IO>
__device__ __forceinline__ float4 load_row4(const IO* p) {
    if constexpr (sizeof(IO) == 4) {
        return __ldg(reinterpret_cast<const float4*>(p));
    } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        const float2 a = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(u.x));
        const float2 b = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
}

// kDots: some call wants its outputs' dot products.  Then outputs come from the decayed state of
// before the token's own update, and its own term (x . y) w joins them after the dot product.
template <int DA, typename IO, bool kOut, bool kDots>
__global__ void __launch_bounds__(128) token_kernel(const __grid_constant__ Problem p,
                                                    const __grid_constant__ Calls calls,
                                                    float* dec,
                                                    int blocks_per_call) {
    constexpr int R = DA / 4, kPer = kTile * DA / 4 / 128, kPerW = kTile * kCols / 4 / 128;
    __shared__ __align__(16) float xs[kOut ? kTile : 1][DA], ys[kTile][DA];
    __shared__ __align__(16) float ws[kDots ? 2 : 1][kTile][kCols];  // (kDots: the last tile's too)
    __shared__ float xy[kTile];  // x . y
    __shared__ float2 fs[kTile];  // how the state decays before the token: factor, near
    __shared__ float2 part[kOut ? 4 : 1][kTile][kCols / 2];
    if (kOut) grid_dependency_wait();
    grid_dependents_launch();
    if (kOut && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) lin::check_seqlens(p);
    const Call& c = calls.c[blockIdx.z / blocks_per_call];
    const int cb = blockIdx.z % blocks_per_call;
    if (c.da != DA || cb * kCols >= c.db) return;
    const Segment sg = lin::find_segment(p, (int)blockIdx.x);
    const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = cb * kCols + 2 * lane, row0 = warp * R;
    const int64_t E = (int64_t)c.da * c.db;
    const int64_t own = ((int64_t)sg.edge * p.H + h) * E;
    const int64_t seq = ((int64_t)sg.n * p.H + h) * E;

    float2 S[2][R / 2];  // [column][row pair]
    auto load_state = [&](const float* from) {
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            const int row = row0 + 2 * r;
            if (from == nullptr) {
                S[0][r] = S[1][r] = make_float2(0.f, 0.f);
            } else if (c.tr) {
                S[0][r] = *reinterpret_cast<const float2*>(from + col * DA + row);
                S[1][r] = *reinterpret_cast<const float2*>(from + (col + 1) * DA + row);
            } else {
                const float2 a = *reinterpret_cast<const float2*>(from + row * c.db + col);
                const float2 b = *reinterpret_cast<const float2*>(from + (row + 1) * c.db + col);
                S[0][r] = make_float2(a.x, b.x);
                S[1][r] = make_float2(a.y, b.y);
            }
        }
    };
    auto store_state = [&](float* to) {
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            const int row = row0 + 2 * r;
            const float2 a = S[0][r], b = S[1][r];
            if (c.tr) {
                *reinterpret_cast<float2*>(to + col * DA + row) = a;
                *reinterpret_cast<float2*>(to + (col + 1) * DA + row) = b;
            } else {
                *reinterpret_cast<float2*>(to + row * c.db + col) = make_float2(a.x, b.x);
                *reinterpret_cast<float2*>(to + (row + 1) * c.db + col) = make_float2(a.y, b.y);
            }
        }
    };
    if (!sg.live) {
        // an empty sequence owns its first slot: its final state is its initial one
        if (kOut && c.S_out && sg.count == 0 && sg.s == 0) {
            load_state(c.edge ? c.edge + seq : nullptr);
            store_state(c.S_out + seq);
        }
        return;
    }
    const bool last = c.reverse ? sg.s == 0 : sg.s == sg.count - 1;
    if (!kOut && last) return;  // no edge state follows from it
    // the edges launch also put the sequence's own edge state into its first slot, so that
    // with S_out in S0's place no segment reads what another has overwritten
    load_state(!kOut ? nullptr : sg.count > 1 ? c.seg + own : c.edge ? c.edge + seq : nullptr);

    const int len = sg.end - sg.begin;
    const int e = threadIdx.x;
    float4 nx[kPer], ny[kPer], nw[kPerW];
    float ng = 0.f, gsum = 0.f;
    // tile t0's rows, in the order of the walk, zeros past its end
    auto load_tile = [&](int t0) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        auto at = [&](int i) { return c.reverse ? sg.end - 1 - t0 - i : sg.begin + t0 + i; };
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = (e + 128 * j) / (DA / 4), d = (e + 128 * j) % (DA / 4) * 4;
            const bool in = t0 + i < len;
            const int64_t t = at(i);
            if (kOut)
                nx[j] = in ? load_row4(static_cast<const IO*>(c.x) + t * c.x_ld + h * DA + d)
                           : zero;
            ny[j] = in ? load_row4(static_cast<const IO*>(c.y) + t * c.y_ld + h * DA + d) : zero;
        }
#pragma unroll
        for (int j = 0; j < kPerW; ++j) {
            const int i = (e + 128 * j) / (kCols / 4), d = (e + 128 * j) % (kCols / 4) * 4;
            nw[j] = t0 + i < len ? load_row4(static_cast<const IO*>(c.w) + at(i) * c.w_ld +
                                             h * c.db + cb * kCols + d)
                                 : zero;
        }
        // reversed, a token's state has decayed by the token's before it in the walk
        if (e < kTile) {
            ng = 0.f;
            if (t0 + e < len && (!c.reverse || t0 + e > 0))
                ng = lin::log_decay(p, at(c.reverse ? e - 1 : e), h);
        }
    };
    auto factor = [](float g) {
        return g > kNear ? make_float2(expm1f(g), 1.f) : make_float2(expf(g), 0.f);
    };
    auto decay = [&](float2 f) {
        const float2 a = make_float2(f.x, f.x);
        if (f.y != 0.f) {
#pragma unroll
            for (int r = 0; r < R / 2; ++r) {
                S[0][r] = fma2(S[0][r], a, S[0][r]);
                S[1][r] = fma2(S[1][r], a, S[1][r]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R / 2; ++r) {
                S[0][r] = mul2(S[0][r], a);
                S[1][r] = mul2(S[1][r], a);
            }
        }
    };
    // outputs of tile t0, of which `part` holds the four warps' shares
    auto write_out = [&](int t0) {
        for (int i = warp; i < min(kTile, len - t0); i += 4) {
            const int64_t t = c.reverse ? sg.end - 1 - t0 - i : sg.begin + t0 + i;
            float2 o = part[0][i][lane];
#pragma unroll
            for (int u = 1; u < 4; ++u) {
                o.x += part[u][i][lane].x;
                o.y += part[u][i][lane].y;
            }
            if (kDots && c.dot) {
                const IO* y = static_cast<const IO*>(c.dot) + t * c.dot_ld + h * c.db + col;
                float x = fmaf(o.x, to_f32(y[0]), o.y * to_f32(y[1]));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                if ((lane & 15) == 0)
                    c.dots[((int64_t)(col / kDotCols) * p.H + h) * p.T + t] = x;
            }
            if (kDots) {
                const float2 w =
                    *reinterpret_cast<const float2*>(&ws[t0 / kTile & 1][i][2 * lane]);
                o = fma2(make_float2(xy[i], xy[i]), w, o);
            }
            IO* to = static_cast<IO*>(c.out) + (t * p.H + h) * c.db + col;
            if constexpr (sizeof(IO) == 4)
                *reinterpret_cast<float2*>(to) = o;
            else
                *reinterpret_cast<__nv_bfloat162*>(to) = __floats2bfloat162_rn(o.x, o.y);
        }
    };
    load_tile(0);
    for (int t0 = 0; t0 < len; t0 += kTile) {
        const int buf = kDots ? t0 / kTile & 1 : 0;
        __syncthreads();
        if (kOut && t0 > 0) write_out(t0 - kTile);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (kOut) reinterpret_cast<float4*>(xs)[e + 128 * j] = nx[j];
            reinterpret_cast<float4*>(ys)[e + 128 * j] = ny[j];
        }
#pragma unroll
        for (int j = 0; j < kPerW; ++j) reinterpret_cast<float4*>(ws[buf])[e + 128 * j] = nw[j];
        if (e < kTile) {
            fs[e] = factor(ng);
            gsum += ng;
        }
        __syncthreads();
        if (t0 + kTile < len) load_tile(t0 + kTile);
        const int m = min(kTile, len - t0);
        if (kDots)
            for (int i = warp; i < m; i += 4) {
                float x = 0.f;
#pragma unroll
                for (int d = lane; d < DA; d += 32) x = fmaf(xs[i][d], ys[i][d], x);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                if (lane == 0) xy[i] = x;
            }
        for (int i = 0; i < m; ++i) {
            decay(fs[i]);
            const float2 w = *reinterpret_cast<const float2*>(&ws[buf][i][2 * lane]);
            const float2 w0 = make_float2(w.x, w.x), w1 = make_float2(w.y, w.y);
            float2 a0 = make_float2(0.f, 0.f), a1 = a0;
            auto read = [&](int r) {
                const float4 x = *reinterpret_cast<const float4*>(&xs[i][row0 + 4 * r]);
                const float2 xa = make_float2(x.x, x.y), xb = make_float2(x.z, x.w);
                a0 = fma2(xa, S[0][2 * r], a0);
                a1 = fma2(xa, S[1][2 * r], a1);
                a0 = fma2(xb, S[0][2 * r + 1], a0);
                a1 = fma2(xb, S[1][2 * r + 1], a1);
            };
#pragma unroll
            for (int r = 0; r < R / 4; ++r) {
                if (kDots) read(r);
                const float4 y = *reinterpret_cast<const float4*>(&ys[i][row0 + 4 * r]);
                const float2 ya = make_float2(y.x, y.y), yb = make_float2(y.z, y.w);
                S[0][2 * r] = fma2(ya, w0, S[0][2 * r]);
                S[1][2 * r] = fma2(ya, w1, S[1][2 * r]);
                S[0][2 * r + 1] = fma2(yb, w0, S[0][2 * r + 1]);
                S[1][2 * r + 1] = fma2(yb, w1, S[1][2 * r + 1]);
                if (kOut && !kDots) read(r);
            }
            if (kOut) part[warp][i][lane] = make_float2(a0.x + a0.y, a1.x + a1.y);
        }
    }
    if (kOut) {
        __syncthreads();
        write_out((len - 1) / kTile * kTile);
    }
    if (c.reverse) {
        const float g = lin::log_decay(p, sg.begin, h);
        decay(factor(g));
        if (e == 0) gsum += g;
    }
    float* to = kOut ? (last && c.S_out ? c.S_out + seq : nullptr)
                     : const_cast<float*>(c.seg) + own;
    if (to) store_state(to);
    if (kDots && last && c.anchor) {
        const float* with = c.anchor + seq;
        float2 x = make_float2(0.f, 0.f);
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            const int row = row0 + 2 * r;
            if (c.tr) {
                x = fma2(S[0][r], *reinterpret_cast<const float2*>(with + col * DA + row), x);
                x = fma2(S[1][r], *reinterpret_cast<const float2*>(with + (col + 1) * DA + row), x);
            } else {
                const float2 a = *reinterpret_cast<const float2*>(with + row * c.db + col);
                const float2 b = *reinterpret_cast<const float2*>(with + (row + 1) * c.db + col);
                x = fma2(S[0][r], make_float2(a.x, b.x), x);
                x = fma2(S[1][r], make_float2(a.y, b.y), x);
            }
        }
        float y = x.x + x.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (lane == 0)
            c.anchors[((int64_t)sg.n * p.H + h) * lin::kAnchors + 4 * cb + warp] = y;
    }
    if (!kOut && cb == 0 && warp == 0) {
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) gsum += __shfl_xor_sync(0xffffffffu, gsum, off);
        if (lane == 0)
            dec[((int64_t)c.reverse * p.edges + sg.edge) * p.H + h] =
                gsum * 1.4426950408889634f;
    }
}

// ------------------------------------------------------------------------ edges --
// A thread carries four state elements over a sequence's segments, the contributions loaded four
// segments ahead, and on to the state after the sequence where the last segment's contribution is
// there (the token kernels form that state themselves).  Bound by that traffic, each contribution
// read and each edge written once, and by its latency where segments are few: 22 us at 65,536
// tokens x 32 heads x 128 (32 segments of 2,048: 134 MB), 43 us for both directions of the
// gradients x 16 heads (64 of 1,024: 268 MB).
struct Edges {
    const float* add[2];    // [edges][H][E] contributions: forward, reversed
    float* seg[2];          // [edges][H][E] edge states (written)
    const float* edge[2];   // [N][H][E] or nullptr
    const float* dec[2];    // [edges][H] summed log2 decays
    float* S_out[2];        // [N][H][E] states after the sequences, or nullptr
    const float* anchor[2];  // as in Call
    float* anchors[2];
    int E;
};

__global__ void __launch_bounds__(256) edge_kernel(const __grid_constant__ Problem p,
                                                   const __grid_constant__ Edges e) {
    constexpr int kAhead = 4;
    grid_dependency_wait();
    grid_dependents_launch();
    const int dir = blockIdx.z;
    const int per_head = e.E / 4 / 256;
    const int h = blockIdx.x / per_head;
    const int at = (blockIdx.x % per_head) * 256 + threadIdx.x;  // float4 within the state
    const int64_t stride = (int64_t)p.H * (e.E / 4), own = (int64_t)h * (e.E / 4) + at;
    const float4* add = reinterpret_cast<const float4*>(e.add[dir]);
    float4* seg = reinterpret_cast<float4*>(e.seg[dir]);
    __shared__ float part[8];
    // sequence n's edges
    auto scan = [&](int n) {
        int64_t a, b;
        seq_range(p.cu, n, p.N, p.T, p.err, a, b);
        const int count = (int)((b - a + p.L - 1) / p.L);
        const int64_t base = lin::edge_base(p, (uint32_t)a, n);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e.edge[dir])
            acc = reinterpret_cast<const float4*>(e.edge[dir])[(int64_t)n * stride + own];
        seg[(base + (dir ? count - 1 : 0)) * stride + own] = acc;
        // step i takes segment s(i)'s contribution and leaves the edge state of segment s(i + 1)
        auto slot = [&](int i) { return base + (dir ? count - 1 - i : i); };
        for (int i0 = 0; i0 < count - 1; i0 += kAhead) {
            float4 in[kAhead];
            float d[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i0 + u < count - 1) {
                    in[u] = __ldcs(add + slot(i0 + u) * stride + own);
                    d[u] = e.dec[dir][slot(i0 + u) * p.H + h];
                }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i0 + u < count - 1) {
                    const float f = exp2f(d[u]);
                    acc.x = fmaf(f, acc.x, in[u].x);
                    acc.y = fmaf(f, acc.y, in[u].y);
                    acc.z = fmaf(f, acc.z, in[u].z);
                    acc.w = fmaf(f, acc.w, in[u].w);
                    seg[slot(i0 + u + 1) * stride + own] = acc;
                }
        }
        if (e.S_out[dir] == nullptr && e.anchor[dir] == nullptr) return;
        const float4 in = __ldcs(add + slot(count - 1) * stride + own);
        const float f = exp2f(e.dec[dir][slot(count - 1) * p.H + h]);
        acc.x = fmaf(f, acc.x, in.x);
        acc.y = fmaf(f, acc.y, in.y);
        acc.z = fmaf(f, acc.z, in.z);
        acc.w = fmaf(f, acc.w, in.w);
        const int64_t at_seq = (int64_t)n * stride + own;
        if (e.S_out[dir]) reinterpret_cast<float4*>(e.S_out[dir])[at_seq] = acc;
        if (e.anchor[dir] == nullptr) return;
        const float4 with = __ldg(reinterpret_cast<const float4*>(e.anchor[dir]) + at_seq);
        float x = fmaf(acc.x, with.x, fmaf(acc.y, with.y, fmaf(acc.z, with.z, acc.w * with.w)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
        __syncthreads();
        // parts by this block and, where a state has fewer blocks than parts, zeros
        float* to = e.anchors[dir] + ((int64_t)n * p.H + h) * lin::kAnchors;
        for (int i = blockIdx.x % per_head; i < lin::kAnchors; i += per_head)
            if (threadIdx.x == 0) {
                x = 0.f;
                if (i < per_head)
                    for (int w = 0; w < 8; ++w) x += part[w];
                to[i] = x;
            }
    };
    __shared__ unsigned some[8];  // of the next 256 sequences of this block's, those with segments
    for (int n0 = blockIdx.y; n0 < p.N; n0 += 256 * gridDim.y) {
        int64_t a = 0, b = 0;
        const int mine = n0 + threadIdx.x * gridDim.y;
        if (mine < p.N) seq_range(p.cu, mine, p.N, p.T, p.err, a, b);
        const unsigned found = __ballot_sync(0xffffffffu, b - a > p.L);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) some[threadIdx.x >> 5] = found;
        __syncthreads();
        for (int w = 0; w < 8; ++w)
            for (unsigned mask = some[w]; mask; mask &= mask - 1)
                scan(n0 + (32 * w + __ffs(mask) - 1) * (int)gridDim.y);
    }
}

// ----------------------------------------------------------- gradient of the decay --
// One CTA a (segment, head): the anchors <S, D> at the segment's two edges, then the prefix sums
// of q.dq - k.dk over its tokens, 256 at a time.  Bound by reading the edge states
// (each anchor's twice, by the segments on both sides): 57 us at 65,536 tokens x 16 heads x 128,
// 268 MB at 4.7 TB/s.
struct DecayGrad {
    const float *segS, *segD;        // [edges][H][E] edge states (where sequences have segments)
    const float *at_start, *at_end;  // [N][H][kAnchors] partial sums of <S, D> at the sequences'
    int n_start, n_end;              //   edges, and how many; nullptr where that is zero
    const float *dots_q, *dots_k;    // [nq][H][T], [nk][H][T]
    int nq, nk;
    float* dg;                       // [T][H]
    int E;
};

__global__ void __launch_bounds__(256) decay_grad_kernel(const __grid_constant__ Problem p,
                                                         const __grid_constant__ DecayGrad d) {
    __shared__ float red[2][8];
    grid_dependency_wait();
    grid_dependents_launch();
    const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Segment sg = lin::find_segment(p, (int)blockIdx.x);
    if (!sg.live) return;
    const int64_t seq = ((int64_t)sg.n * p.H + h) * lin::kAnchors;
    const int64_t own = ((int64_t)sg.edge * p.H + h) * d.E, step = (int64_t)p.H * d.E;
    auto dot = [&](const float* A, const float* B) {
        float x = 0.f;
#pragma unroll 8
        for (int i = threadIdx.x; i < d.E / 4; i += 256) {
            const float4 u = reinterpret_cast<const float4*>(A)[i];
            const float4 v = reinterpret_cast<const float4*>(B)[i];
            x = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, x))));
        }
        return x;
    };
    auto part = [&](const float* parts, int n) {
        return parts && (int)threadIdx.x < n ? parts[seq + threadIdx.x] : 0.f;
    };
    // sums of x and of y over the block, the same in every thread
    auto block_sum = [&](float& x, float& y) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, off);
            y += __shfl_xor_sync(0xffffffffu, y, off);
        }
        __syncthreads();
        if (lane == 0) { red[0][warp] = x; red[1][warp] = y; }
        __syncthreads();
        x = y = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) { x += red[0][w]; y += red[1][w]; }
    };
    // segment s's slot holds S at its start and D at its end
    const bool first = sg.s == 0, last = sg.s == sg.count - 1;
    float head = first ? part(d.at_start, d.n_start) : dot(d.segS + own, d.segD + own - step);
    float tail = last ? part(d.at_end, d.n_end) : dot(d.segS + own + step, d.segD + own);
    block_sum(head, tail);
    auto term = [&](int64_t t, float& x, float& size) {
        x = size = 0.f;
        if (t >= sg.end) return;
        float a = 0.f, b = 0.f;
        for (int i = 0; i < d.nq; ++i) a += d.dots_q[((int64_t)i * p.H + h) * p.T + t];
        for (int i = 0; i < d.nk; ++i) b += d.dots_k[((int64_t)i * p.H + h) * p.T + t];
        x = a - b;
        size = fabsf(a) + fabsf(b);
    };
    // the sum over the block's threads before this one, and over all
    auto scan = [&](float x, float (&warps)[8], float& before, float& all) {
        float y = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float z = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) y += z;
        }
        if (lane == 31) warps[warp] = y;
        __syncthreads();
        before = all = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) before += warps[w];
            all += warps[w];
        }
        y = __shfl_up_sync(0xffffffffu, y, 1);
        if (lane > 0) before += y;
    };
    // The miss is that of the sums as they will be taken: added up in another order, they would end
    // elsewhere by their rounding.
    float sum = 0.f, weight = 0.f;
    for (int64_t t0 = sg.begin; t0 < sg.end; t0 += 256) {
        float x, size, before, all;
        term(t0 + threadIdx.x, x, size);
        __syncthreads();
        scan(x, red[0], before, all);
        sum += all;
        weight = fmaf(size, size, weight);
    }
    float none = 0.f;
    block_sum(weight, none);
    const float miss = (tail - head) + sum;
    const float share = weight > 0.f && weight < INFINITY ? miss / weight : 0.f;
    sum = weight = 0.f;
    for (int64_t t0 = sg.begin; t0 < sg.end; t0 += 256) {
        const int64_t t = t0 + threadIdx.x;
        float x, size, before, all, back, backs;
        term(t, x, size);
        __syncthreads();
        scan(x, red[0], before, all);
        scan(size * size, red[1], back, backs);
        if (t < sg.end) d.dg[t * p.H + h] = head - ((sum + before) - share * (weight + back));
        sum += all;
        weight += backs;
    }
}

// dg of a decay that all tokens of a head share: the sum over tokens, in a fixed order, by one CTA
// a head.  Bound by its rounds' latency: 24 us at 65,536 tokens x 16 heads, 2 % of the gradients.
__global__ void __launch_bounds__(256) decay_sum_kernel(const float* dg, int64_t T, int H,
                                                        float* out) {
    __shared__ float red[256];
    grid_dependency_wait();
    const int h = blockIdx.x;
    float x = 0.f;
    for (int64_t t = threadIdx.x; t < T; t += 256) x += dg[t * H + h];
    red[threadIdx.x] = x;
    for (int n = 128; n > 0; n >>= 1) {
        __syncthreads();
        if (threadIdx.x < n) red[threadIdx.x] += red[threadIdx.x + n];
    }
    if (threadIdx.x == 0) out[h] = red[0];
}

// ------------------------------------------------------------------------- host --

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// bf16 runs on the tensor cores, fp32 (whose operands they would round) token by token.
// KDA_FWD_PATH=generic in the environment forces the latter (the tests cross-check the two).
bool use_tc(int io_bf16) {
    const char* env = getenv("KDA_FWD_PATH");
    return io_bf16 && !(env && strcmp(env, "generic") == 0);
}

// Tokens a segment.  On the tensor cores a segment's chunks in a row cost less than its edge states
// (two fp32 states a segment, written, read and loaded), so segments are as long as they can be and
// still be one for every SM, or for half of the SMs where the next length down would give more than
// one to each: at 8,192 tokens x 16 heads 128 segments of 1,024 tokens take 89 us, 256 of 512 take
// 95, 512 of 256 take 110; x 10 heads 80 of 1,024 take 79, 160 of 512 take 87.  Not beyond 2,048
// tokens, where the last round's ends cost more (65,536 x 32: 824 us, with 4,096 882, with 1,024
// 892; packed prompts up to 5,753 tokens x 16, whose lengths the rule does not know: 353, 403,
// 337); in the gradients not beyond 1,024, for the rounding between two anchors adds up in dg
// (65,536 x 16: 2.0e-6 off, with 2,048 2.4e-6 and 1,455 instead of 1,515 us).  Up to 256 tokens
// take no segments: two chunks in a row take about as long as the edges' launch (256 x 4: 30
// against 28 us, and one launch less for the host; 512 x 4 in one piece 42 against 30, its
// gradients 71 against 50). Token by token a segment is walked by as many CTAs as its state has
// blocks, and each SM needs several to be busy: four segments an SM (2,048 + 1,531 tokens x 8
// heads: 77 us, two 89, one 138).
int segment_length(int64_t T, int H, bool tc, bool bwd) {
    if (tc && T <= 256) return 256;
    int L = tc ? 128 : 64;
    const int most = tc && !bwd ? 2048 : 1024, fill = tc ? 152 : 4 * 152;
    while (L < most && T / L * H > fill) L *= 2;
    return L;
}

struct Layout {
    int L;
    int64_t slots, edges;
    bool segments;  // some sequence may be longer than a segment
    size_t rec, next, add[2], seg[2], dec, at_start, at_end, dots_q, dots_k, dg, bytes;
};

Layout layout(int64_t T, int N, int H, int dk, int dv, bool bwd, bool tc, bool equal) {
    Layout l{};
    l.L = segment_length(T, H, tc, bwd);
    l.slots = lin::slot_count(T, N, l.L);
    l.edges = std::min(l.slots, 2 * T / l.L);
    l.segments = (equal && N > 0 ? T / N : T) > l.L;
    const size_t state = (size_t)H * dk * dv * sizeof(float);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += align256(n);
        return r;
    };
    l.rec = take(tc ? lintc::record_bytes(T, N, H) : 0);
    l.next = take(tc ? lintc::kCounters * sizeof(unsigned) : 0);
    for (int i = 0; i < (bwd ? 2 : 1); ++i) {
        l.add[i] = take(l.segments ? (size_t)l.edges * state : 0);
        l.seg[i] = take(l.segments ? (size_t)l.edges * state : 0);
    }
    l.dec = take(l.segments ? (size_t)2 * l.edges * H * sizeof(float) : 0);
    if (bwd) {
        l.at_start = take((size_t)N * H * lin::kAnchors * sizeof(float));
        l.at_end = take((size_t)N * H * lin::kAnchors * sizeof(float));
        l.dots_q = take((size_t)(dk / kDotCols) * T * H * sizeof(float));
        l.dots_k = take((size_t)(dk / kDotCols) * T * H * sizeof(float));
        l.dg = take((size_t)T * H * sizeof(float));
    }
    l.bytes = at;
    return l;
}

Problem problem(const LinearArgs& a, const Layout& l) {
    Problem p{};
    p.cu = a.cu_seqlens; p.N = a.N; p.T = a.T_total; p.H = a.H; p.g = a.g;
    p.g_per_token = a.g_per_token; p.L = l.L; p.edges = (int)l.edges;
    p.edges_close = l.edges < l.slots; p.err = a.dev_err;
    return p;
}

template <typename IO, bool kOut, bool kDots>
cudaError_t launch_token(const Problem& p, const Calls& calls, int n, int64_t slots, float* dec,
                         const char* name, cudaStream_t s) {
    const int blocks = 128 / kCols;
    const dim3 grid((unsigned)slots, p.H, n * blocks);
    bool any[2] = {};
    for (int i = 0; i < n; ++i) any[calls.c[i].da == 128] = true;
    const auto k64 = token_kernel<64, IO, kOut, kDots>, k128 = token_kernel<128, IO, kOut, kDots>;
    ProfScope prof(name, s);
    cudaError_t e = cudaSuccess;
    if (!kOut) {  // (a call's first launch, one da for both directions)
        if (any[0]) k64<<<grid, 128, 0, s>>>(p, calls, dec, blocks);
        if (any[1]) k128<<<grid, 128, 0, s>>>(p, calls, dec, blocks);
        return cudaGetLastError();
    }
    if (any[0]) e = launch_dependent(k64, grid, 128, 0, s, p, calls, dec, blocks);
    if (any[1] && e == cudaSuccess)
        e = launch_dependent(k128, grid, 128, 0, s, p, calls, dec, blocks);
    return e;
}

template <typename IO, bool kOut>
cudaError_t launch_token(const Problem& p, const Calls& calls, int n, int64_t slots, float* dec,
                         const char* name, cudaStream_t s) {
    bool dots = false;
    for (int i = 0; i < n; ++i) dots = dots || calls.c[i].dot != nullptr;
    return kOut && dots ? launch_token<IO, kOut, kOut>(p, calls, n, slots, dec, name, s)
                        : launch_token<IO, kOut, false>(p, calls, n, slots, dec, name, s);
}

struct Scratch {  // of the workspace
    uint8_t* ws;
    Layout l;
    float* at(size_t off) const { return reinterpret_cast<float*>(ws + off); }
    const float* rec() const { return at(l.rec); }
    unsigned* next(int i) const { return reinterpret_cast<unsigned*>(ws + l.next) + i; }
};

// The outputs of some calls.
cudaError_t launch_out(const LinearArgs& a, const Problem& p, const Scratch& w, const Calls& calls,
                       int n, const char* name) {
    if (use_tc(a.io_bf16)) {
        // (calls with dot products and the others are kernels of their own)
        int m = 0;
        while (m < n && calls.c[m].dot) ++m;
        Calls rest{};
        for (int i = m; i < n; ++i) rest.c[i - m] = calls.c[i];
        if (m > 0)
            if (cudaError_t e = lintc::launch_outputs(p, calls, m, w.l.slots, w.rec(), w.next(0),
                                                      name, a.stream))
                return e;
        return m == n ? cudaSuccess
                      : lintc::launch_outputs(p, rest, n - m, w.l.slots, w.rec(),
                                              w.next(m > 0 ? 2 : 0), name, a.stream);
    }
    return a.io_bf16 ? launch_token<__nv_bfloat16, true>(p, calls, n, w.l.slots, nullptr, name,
                                                         a.stream)
                     : launch_token<float, true>(p, calls, n, w.l.slots, nullptr, name, a.stream);
}

// Segment sums, edge states and (on the tensor cores) final states of the forward states and, in a
// backward pass, of the reversed ones; `calls` has their rows and what is wanted at the end.
cudaError_t launch_states(const LinearArgs& a, const Problem& p, const Scratch& w, Calls calls,
                          int n, int sums, int counter) {
    const bool tc = use_tc(a.io_bf16);
    bool final = false;
    for (int i = 0; i < n; ++i) final = final || calls.c[i].S_out || calls.c[i].anchor;
    if (!w.l.segments) sums &= ~lintc::kSegments;
    if (!tc || !final) sums &= ~lintc::kSingles;
    if (sums == 0) return cudaSuccess;
    float* dec = w.at(w.l.dec);
    Edges e{};
    for (int i = 0; i < n; ++i) {
        Call& c = calls.c[i];
        c.seg = w.at(w.l.add[i]);
        e.add[i] = c.seg;
        e.seg[i] = w.at(w.l.seg[i]);
        e.edge[i] = c.edge;
        e.dec[i] = dec + (size_t)i * w.l.edges * a.H;
        if (tc) {
            e.S_out[i] = c.S_out;
            e.anchor[i] = c.anchor;
            e.anchors[i] = c.anchors;
        }
    }
    e.E = a.dk * a.dv;
    const char* name = sums & lintc::kSegments ? "linear_segment_kernel" : "linear_state_kernel";
    cudaError_t err =
        tc ? lintc::launch_sums(p, calls, n, w.l.slots, w.rec(), dec, w.next(counter), sums, name,
                                a.stream)
        : a.io_bf16
            ? launch_token<__nv_bfloat16, false>(p, calls, n, w.l.slots, dec, name, a.stream)
            : launch_token<float, false>(p, calls, n, w.l.slots, dec, name, a.stream);
    if (err != cudaSuccess || !(sums & lintc::kSegments)) return err;
    ProfScope prof("linear_edge_kernel", a.stream);
    const int per_row = a.H * (e.E / 1024), most = std::max(1, 8 * 8 * 152 / per_row);
    const dim3 grid(per_row, std::min(a.N, most), n);
    return launch_dependent(edge_kernel, grid, dim3(256), 0, a.stream, p, e);
}

cudaError_t launch_decays(const LinearArgs& a, const Problem& p, const Scratch& w) {
    if (!use_tc(a.io_bf16)) return cudaSuccess;
    return lintc::launch_decays(p, w.at(w.l.rec), w.next(0), a.stream);
}

}  // namespace

size_t linear_fwd_workspace_size(int64_t T, int N, int H, int dk, int dv, int io_bf16) {
    return layout(T, N, H, dk, dv, false, use_tc(io_bf16), false).bytes;
}
size_t linear_bwd_workspace_size(int64_t T, int N, int H, int dk, int dv, int io_bf16) {
    return layout(T, N, H, dk, dv, true, use_tc(io_bf16), false).bytes;
}

cudaError_t launch_linear_fwd(const LinearArgs& a) {
    const Scratch w{static_cast<uint8_t*>(a.workspace),
                    layout(a.T_total, a.N, a.H, a.dk, a.dv, false, use_tc(a.io_bf16),
                           a.cu_seqlens == nullptr)};
    const Problem p = problem(a, w.l);
    if (cudaError_t e = launch_decays(a, p, w)) return e;
    Calls calls{};
    Call& c = calls.c[0];
    c.x = a.q; c.x_ld = a.q_ld; c.y = a.k; c.y_ld = a.k_ld; c.w = a.v; c.w_ld = a.v_ld;
    c.da = a.dk; c.db = a.dv; c.edge = a.S0; c.S_out = a.S_out; c.out = a.o;
    // With S_out in S0's place the states after sequences of one segment come after the outputs,
    // which read S0 itself there.
    const bool in_place = a.S_out != nullptr && a.S_out == a.S0;
    const int first = lintc::kSegments | (in_place ? 0 : lintc::kSingles);
    if (cudaError_t e = launch_states(a, p, w, calls, 1, first, 1)) return e;
    c.seg = w.l.segments ? w.at(w.l.seg[0]) : nullptr;
    if (cudaError_t e = launch_out(a, p, w, calls, 1, "linear_out_kernel")) return e;
    return in_place ? launch_states(a, p, w, calls, 1, lintc::kSingles, 2) : cudaSuccess;
}

cudaError_t launch_linear_bwd(const LinearArgs& a) {
    const Scratch w{static_cast<uint8_t*>(a.workspace),
                    layout(a.T_total, a.N, a.H, a.dk, a.dv, true, use_tc(a.io_bf16),
                           a.cu_seqlens == nullptr)};
    const Layout& l = w.l;
    const Problem p = problem(a, l);
    if (cudaError_t e = launch_decays(a, p, w)) return e;
    Calls states{};  // S from the starts, D from the ends
    Call &S = states.c[0], &D = states.c[1];
    S.y = a.k; S.y_ld = a.k_ld; S.w = a.v; S.w_ld = a.v_ld; S.edge = a.S0;
    D.y = a.q; D.y_ld = a.q_ld; D.w = a.dout; D.w_ld = a.dout_ld; D.edge = a.dS_out;
    S.da = D.da = a.dk; S.db = D.db = a.dv; D.reverse = 1; D.S_out = a.dS0;
    if (a.dg) {
        S.anchor = a.dS_out; S.anchors = w.at(l.at_end);
        D.anchor = a.S0; D.anchors = w.at(l.at_start);
    }
    if (cudaError_t e =
            launch_states(a, p, w, states, 2, lintc::kSegments | lintc::kSingles, 1))
        return e;
    float* const seg[2] = {l.segments ? w.at(l.seg[0]) : nullptr,
                           l.segments ? w.at(l.seg[1]) : nullptr};
    Calls calls{};
    Call &q = calls.c[0], &k = calls.c[1], &v = calls.c[2];
    q.x = a.dout; q.x_ld = a.dout_ld; q.y = a.v; q.y_ld = a.v_ld; q.w = a.k; q.w_ld = a.k_ld;
    q.da = a.dv; q.db = a.dk; q.tr = 1; q.edge = a.S0; q.seg = seg[0]; q.out = a.dq;
    k.x = a.v; k.x_ld = a.v_ld; k.y = a.dout; k.y_ld = a.dout_ld; k.w = a.q; k.w_ld = a.q_ld;
    k.da = a.dv; k.db = a.dk; k.reverse = 1; k.tr = 1; k.edge = a.dS_out; k.seg = seg[1];
    k.out = a.dk_;
    v.x = a.k; v.x_ld = a.k_ld; v.y = a.q; v.y_ld = a.q_ld; v.w = a.dout; v.w_ld = a.dout_ld;
    v.da = a.dk; v.db = a.dv; v.reverse = 1; v.edge = a.dS_out; v.seg = seg[1]; v.out = a.dv_;
    v.S_out = a.dS0;
    if (a.dg) {
        q.dot = a.q; q.dot_ld = a.q_ld; q.dots = w.at(l.dots_q);
        k.dot = a.k; k.dot_ld = a.k_ld; k.dots = w.at(l.dots_k);
        q.anchor = S.anchor; q.anchors = S.anchors;
        v.anchor = D.anchor; v.anchors = D.anchors;
    }
    if (cudaError_t e = launch_out(a, p, w, calls, 3, "linear_grad_kernel")) return e;
    if (a.dg) {
        DecayGrad d{};
        d.segS = seg[0]; d.segD = seg[1];
        // (the tensor cores' kernels leave 16 parts, the other four a 64 columns)
        const bool tc = use_tc(a.io_bf16);
        d.at_start = a.S0 ? D.anchors : nullptr; d.n_start = tc ? lin::kAnchors : a.dv / kCols * 4;
        d.at_end = a.dS_out ? S.anchors : nullptr; d.n_end = tc ? lin::kAnchors : a.dk / kCols * 4;
        d.dots_q = q.dots; d.dots_k = k.dots; d.nq = d.nk = a.dk / kDotCols;
        d.dg = a.g_per_token ? a.dg : w.at(l.dg); d.E = a.dk * a.dv;
        if (a.T_total > 0) {
            ProfScope prof("linear_decay_grad_kernel", a.stream);
            if (cudaError_t err = launch_dependent(decay_grad_kernel,
                                                   dim3((unsigned)l.slots, a.H), dim3(256), 0,
                                                   a.stream, p, d))
                return err;
        }
        if (!a.g_per_token) {
            ProfScope prof("linear_decay_sum_kernel", a.stream);
            if (cudaError_t err = launch_dependent(decay_sum_kernel, dim3(a.H), dim3(256), 0,
                                                   a.stream, (const float*)d.dg, a.T_total, a.H,
                                                   a.dg))
                return err;
        }
    }
    return cudaGetLastError();
}

// ------------------------------------------------------------------------ decode --
// One CTA a (request, head): a state row of dv fp32 is covered by dv / 4 lanes with a float4
// each, the dk rows spread over 8 warps; every element is read once, updated, written once and
// added to its column's output:  S <- e^g S + k v^T,  o = S^T q.
// Bound by the states, once in and once out: 256 requests x 32 heads x 128 x 128 take 158 us,
// 1.07 GB at 6.8 TB/s, the copy rate.  A few requests: 10 us, the latency of one CTA.
namespace {

template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(256) step_kernel(const IO* __restrict__ q, int64_t q_ld,
                                                   const IO* __restrict__ k, int64_t k_ld,
                                                   const IO* __restrict__ v, int64_t v_ld,
                                                   const float* __restrict__ g, int g_per_token,
                                                   float* __restrict__ S,
                                                   const int32_t* __restrict__ slots, int n_slots,
                                                   int H, IO* __restrict__ o, unsigned* err) {
    constexpr int kLanesPerRow = DV / 4;
    constexpr int kRowsPerPass = 256 / kLanesPerRow;
    constexpr int kRows = DK / kRowsPerPass;
    __shared__ float s_k[DK], s_q[DK];
    __shared__ float4 s_red[8][kLanesPerRow];
    const int n = blockIdx.x / H, h = blockIdx.x % H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid % kLanesPerRow, row0 = tid / kLanesPerRow;
    const int slot = slots ? __ldg(slots + n) : n;
    if (slot < 0 || slot >= n_slots) {
        if (slot >= n_slots && tid == 0) atomicOr(err, kDevErrBadSlot);
        if (tid < DV) o[(size_t)blockIdx.x * DV + tid] = from_f32<IO>(0.f);
        return;
    }
    float4* Sp = reinterpret_cast<float4*>(S + ((size_t)slot * H + h) * DK * DV);
    float4 s[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m)
        s[m] = __ldcs(Sp + (row0 + m * kRowsPerPass) * kLanesPerRow + col);
    const float a = expf(g_per_token ? __ldg(g + blockIdx.x) : __ldg(g + h));
    for (int c = tid; c < DK; c += 256) {
        s_k[c] = to_f32(k[n * k_ld + h * DK + c]);
        s_q[c] = to_f32(q[n * q_ld + h * DK + c]);
    }
    const IO* vp = v + n * v_ld + h * DV + 4 * col;
    const float4 w = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        const int row = row0 + m * kRowsPerPass;
        const float kr = s_k[row], qr = s_q[row];
        float4 r;
        r.x = fmaf(a, s[m].x, kr * w.x);
        r.y = fmaf(a, s[m].y, kr * w.y);
        r.z = fmaf(a, s[m].z, kr * w.z);
        r.w = fmaf(a, s[m].w, kr * w.w);
        __stcs(Sp + row * kLanesPerRow + col, r);
        acc.x = fmaf(qr, r.x, acc.x);
        acc.y = fmaf(qr, r.y, acc.y);
        acc.z = fmaf(qr, r.z, acc.z);
        acc.w = fmaf(qr, r.w, acc.w);
    }
    if (kLanesPerRow < 32) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
    }
    if (lane < kLanesPerRow) s_red[warp][lane] = acc;
    __syncthreads();
    if (tid < DV) {
        float x = 0.f;
#pragma unroll
        for (int w8 = 0; w8 < 8; ++w8) x += reinterpret_cast<const float*>(s_red[w8])[tid];
        o[(size_t)blockIdx.x * DV + tid] = from_f32<IO>(x);
    }
}

struct StepArgs {
    const void *q, *k, *v;
    int64_t q_ld, k_ld, v_ld;
    const float* g;
    int g_per_token;
    float* S;
    const int32_t* slots;
    int n_slots, N, H;
    void* o;
    unsigned* err;
    cudaStream_t stream;
};

template <int DK, int DV, typename IO>
cudaError_t step_t(const StepArgs& a) {
    ProfScope prof("linear_step_kernel", a.stream);
    step_kernel<DK, DV, IO><<<a.N * a.H, 256, 0, a.stream>>>(
        static_cast<const IO*>(a.q), a.q_ld, static_cast<const IO*>(a.k), a.k_ld,
        static_cast<const IO*>(a.v), a.v_ld, a.g, a.g_per_token, a.S, a.slots, a.n_slots, a.H,
        static_cast<IO*>(a.o), a.err);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t step_dims(const StepArgs& a, int dk, int dv) {
    if (dk == 128) return dv == 128 ? step_t<128, 128, IO>(a) : step_t<128, 64, IO>(a);
    return dv == 128 ? step_t<64, 128, IO>(a) : step_t<64, 64, IO>(a);
}

}  // namespace

cudaError_t launch_linear_decode(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                 const void* v, int64_t v_ld, const float* g, int g_per_token,
                                 float* S, const int32_t* slots, int n_slots, int N, int H, int dk,
                                 int dv, int io_bf16, void* o, unsigned* dev_err,
                                 cudaStream_t stream) {
    const StepArgs a{q, k, v, q_ld, k_ld, v_ld, g, g_per_token, S, slots, n_slots, N, H, o,
                     dev_err, stream};
    return io_bf16 ? step_dims<__nv_bfloat16>(a, dk, dv) : step_dims<float>(a, dk, dv);
}

}  // namespace kda
