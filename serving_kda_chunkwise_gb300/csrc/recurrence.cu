// recurrence.cu -- the gated recurrence of single channels (declared in include/kda.h): packed
// forward, gradients (from whole or 8-bit inputs) and the single-token step.
//
//   h_t = a_t h_{t-1} + b_t,   a = e^g, b = sqrt(1 - e^{2g}) s(i) x           (recurrence_math.cuh)
//   l_t = dy_t + a_{t+1} l_{t+1}, backwards, for the gradients
//
// Both are scans of affine maps (P, H): h -> P h + H.  A cluster of CTAs takes 64 channels along a
// run, some consecutive sequences.  In a step each of its CTAs has a tile of 64 or 128 tokens: each of
// eight warps holds 8 or 16 tokens, a lane two channels, and leaves its tokens' map in shared memory.
// Two warps, a lane a channel, compose the maps, send the tile's to every CTA of the cluster (stores
// into distributed shared memory that count their bytes on a barrier there) and carry the state over
// the cluster's maps; then every warp goes over its tokens again, in registers, and writes.  So inputs
// are read once (by the copy engine, steps ahead), results written once, in rows of 128 bytes (bf16),
// and no cluster waits for another.  Ways that were slower at 65,536 x 4096 (now 443 us): a look-back
// over tiles by messages in memory, 890 us; columns of 16 channels without clusters, 715 us, for the
// copies of 32-byte rows; 8 tokens a warp instead of 16, 531 us; CTAs of 4 or 16 warps, 580 and 880 us.
//
// The gradients go over the tiles backwards.  A thread's states come from the edges, the state that
// every 8th token starts from, which the forward writes on request; without them a forward that
// writes nothing else runs first.  So the factors of l_t in the gradients are formed once, before
// the scan, and stay in registers until l_t is known (which is why a warp has 8 tokens).
//
// Bound by instructions (two a cycle and SM, of which the pairs' take two cycles), by the exchange
// between a step's two passes, and by the clusters' being 256 CTAs for 152 SMs: the forward of
// 65,536 x 4096 in bf16 443 us, 4.8 TB/s (its special functions alone would be 190 us, its memory 322);
// gradients from edges of 32,768 x 4096 430 us, 120 instructions for two channels of a token; from
// 8-bit inputs of 65,536 x 2048 257 us for the edges and 522 us.  (Spills within the steps cost much,
// for tiles leave the first-level cache nothing: 12 bytes 1,610 us.  The 4 bytes that the compiler
// spills of the gradients from 8-bit inputs do not show: without them 524 us.)
//
// Sequences: a setup launch finds the tokens with which sequences start and end, 8 at a time, and
// cuts the batch into runs (one sequence needs none of it, and short forwards of a few do it
// themselves).  Where a sequence starts, a map is constant, which is said by a P that is none, and
// selected, not multiplied by zero, so that nothing that is not finite crosses.
//
// Of several tokens' decay P next to one, P - 1 is kept and composed (a number <= 0), from the tokens'
// summed gates: P's rounding, the same again and again under gates that are alike, would add up over
// the memory (5.7e-6 of a state that remembers 1,600 tokens, now 1e-6; that is 4 % of the forward's time).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "kda_internal.h"
#include "recurrence_math.cuh"
#include "tc_util.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kEdge = 8;    // tokens from one edge to the next, and of a word of marks
constexpr int kC = 64;      // channels of a tile, and of an exponent of packed inputs
constexpr int kWarps = 8;
constexpr int kMaxCluster = 8;
constexpr int kThreads = 32 * kWarps;

// Sequences that a CTA of the scan finds its way through by itself, a lane of a warp each.
constexpr int kFew = 32, kNone = 0x7fffffff;

// What the setup launch leaves for the scan.
struct Plan {
    int* run;            // [runs + 1] first tokens; nullptr, as all here, without it
    uint32_t* marks;     // [ceil(T / 8)] bits of tokens that start (0..7) and end (8..15) a sequence
    int *start_seq, *end_seq;  // [T] whose sequence, at such tokens
    int runs, cols;
    bool few;  // a few sequences, without a setup launch
};

// ---------------------------------------------------------------- inputs --

// The tensors as the copy engine sees them, boxes of a tile's tokens x 64 channels: inputs x, z, i, dy and
// outputs y, or dx, dz and di.
struct Tensors {
    CUtensorMap in[4], out[3];
    int plain;  // inputs by plain copies: rows of codes that begin on 8 bytes only
};

// A stage of the ring: the inputs of a tile, kTok tokens a warp.  The gradients' results leave from where its inputs were, or
// from a place of their own where these have fewer bytes.
template <typename In, typename IO, bool kBwd, int kTok_>
struct Stage {
    static constexpr int kTok = kTok_, kT = kTok * kWarps;
    static constexpr int kIn = kT * kC * (int)sizeof(In), kOut = kT * kC * (int)sizeof(IO);
    static constexpr int kDy = 3 * kIn;
    static constexpr int kExps = kDy + (kBwd ? kOut : 0);
    static constexpr int kBytes = (kExps + (sizeof(In) == 1 ? 3 * kT * 4 : 0) + 127) / 128 * 128;
    static constexpr bool kInPlace = sizeof(In) == sizeof(IO);
    static constexpr int kOuts = kInPlace ? 0 : 3 * kOut;  // bytes of that place
};

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
}

// kT tokens x 64 channels of a tensor by a warp's plain copies; rows and channels past its end become
// zeros.
template <typename In, int kT>
__device__ __forceinline__ void copy_tile(char* dst, const void* src, int64_t ld, int64_t t0, int c0,
                                          int64_t T, int D, int lane) {
    constexpr int kElems = 8 / (int)sizeof(In);
    for (int p = lane; p < kT * kC / kElems; p += 32) {
        const int row = p * kElems / kC, c = p * kElems % kC;
        const bool live = t0 + row < T && c0 + c < D;
        const In* s = static_cast<const In*>(src) + (live ? (t0 + row) * ld + c0 + c : 0);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(
                         smem_u32(dst) + (row * kC + c) * (int)sizeof(In)),
                     "l"(s), "r"(live ? 8 : 0));
    }
}

// Arrivals that fill a stage: the copies' (every lane's where they are plain ones), and for packed
// inputs that of the exponents.
template <typename In>
__device__ __forceinline__ int fill_count(const Tensors& m) {
    return sizeof(In) == 1 ? 1 + (m.plain ? 32 : 1) : 1;
}
// A lane's share of a tile's exponents, on their way.
template <int kT>
struct Exps {
    int8_t e[3 * kT / 32];
};

// Starts the loads of the tile from token t0 and channel c0; called by a warp.
template <typename S, typename In, typename IO, bool kBwd>
__device__ __forceinline__ void load_stage(const RecurrenceArgs& a, const Tensors& m, char* st,
                                           uint64_t* full, int t0, int c0, int lane,
                                           Exps<S::kT>& exps) {
    if (sizeof(In) == 1 && m.plain) {
        copy_tile<In, S::kT>(st, a.x, a.x_ld, t0, c0, a.T_total, a.D, lane);
        copy_tile<In, S::kT>(st + S::kIn, a.z, a.z_ld, t0, c0, a.T_total, a.D, lane);
        copy_tile<In, S::kT>(st + 2 * S::kIn, a.i, a.i_ld, t0, c0, a.T_total, a.D, lane);
        if (kBwd) copy_tile<IO, S::kT>(st + S::kDy, a.dy, a.dy_ld, t0, c0, a.T_total, a.D, lane);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full))
                     : "memory");
    } else if (lane == 0) {
        mbar_expect_tx(full, S::kExps);
        tma_load(st, &m.in[0], c0, t0, full);
        tma_load(st + S::kIn, &m.in[1], c0, t0, full);
        tma_load(st + 2 * S::kIn, &m.in[2], c0, t0, full);
        if (kBwd) tma_load(st + S::kDy, &m.in[3], c0, t0, full);
    }
    if (sizeof(In) == 1) {
#pragma unroll
        for (int j = 0; j < 3 * S::kT / 32; ++j) {
            const int n = j * 32 + lane, t = n % S::kT;
            const int8_t* e = n < S::kT ? a.x_exps : n < 2 * S::kT ? a.z_exps : a.i_exps;
            exps.e[j] = t0 + t < a.T_total ? __ldg(e + (int64_t)(c0 / kC) * a.T_total + t0 + t) : 0;
        }
    }
}
// Puts the powers of two into the stage that load_stage was called for.
template <typename S, typename In>
__device__ __forceinline__ void put_exps(char* st, uint64_t* full, int lane,
                                         const Exps<S::kT>& exps) {
    if (sizeof(In) == 1) {
#pragma unroll
        for (int j = 0; j < 3 * S::kT / 32; ++j)
            // 2^e, denormal at -127; -128 stands for NaN
            reinterpret_cast<float*>(st + S::kExps)[j * 32 + lane] = __int_as_float(
                exps.e[j] > -127 ? (exps.e[j] + 127) << 23 : exps.e[j] == -127 ? 1 << 22 : 0x7fc00000);
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
    }
}

__device__ __forceinline__ float2 bits(__nv_bfloat162 v) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&v);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair(const __nv_bfloat16* p) {
    // (read as what it is: results are written to the same places)
    return bits(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ float2 pair(const float* p) {
    return *reinterpret_cast<const float2*>(p);
}

// A thread's view of a stage: token k of its warp, its two channels.
template <typename S, typename In, typename IO>
struct View {
    char *st, *outs;
    int warp, lane;
    template <typename E>
    __device__ __forceinline__ const E* at(int part, int k) const {
        return reinterpret_cast<const E*>(st + part) + (warp * S::kTok + k) * kC + 2 * lane;
    }
    __device__ __forceinline__ float2 input(int which, int k) const {
        const In* p = at<In>(which * S::kIn, k);
        if constexpr (sizeof(In) == 1) {
            const float s =
                reinterpret_cast<const float*>(st + S::kExps)[which * S::kT + warp * S::kTok + k];
            // a byte with its sign flipped, code + 128, as the last of a number of 2^23 and more
            const uint32_t q = *reinterpret_cast<const uint16_t*>(p) ^ 0x8080u;
            return mul_pair(add_pair(make_float2(__uint_as_float(__byte_perm(q, 0x4b000000u, 0x7440)),
                                                 __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7441))),
                                     both(-8388736.f)),
                            both(s));
        } else {
            return pair(p);
        }
    }
    // The same, infinities as the largest numbers (beside a gradient of zero: its share is zero).
    __device__ __forceinline__ float2 finite(int which, int k) const {
        if constexpr (sizeof(In) == 1) {
            return input(which, k);
        } else if constexpr (sizeof(In) == 2) {
            const __nv_bfloat162 top = __floats2bfloat162_rn(3.3e38f, 3.3e38f);
            const __nv_bfloat162 v =
                __hmin2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(at<In>(which * S::kIn, k)),
                                __hneg2(top)),
                        top);
            return bits(v);
        } else {
            const float2 v = input(which, k);
            return make_float2(fminf(fmaxf(v.x, -3e38f), 3e38f), fminf(fmaxf(v.y, -3e38f), 3e38f));
        }
    }
    __device__ __forceinline__ float2 dy(int k) const { return pair(at<IO>(S::kDy, k)); }
    // the place of result `which` of token k
    __device__ __forceinline__ IO* out(int which, int k) const {
        return reinterpret_cast<IO*>(outs + which * S::kOut) + (warp * S::kTok + k) * kC + 2 * lane;
    }
};

__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void store_pair(float* p, float2 v) {
    *reinterpret_cast<float2*>(p) = v;
}
// Two channels of row n of an fp32 [N, D] tensor.
__device__ __forceinline__ float2 state_row(const float* p, int n, int D, int c) {
    return *reinterpret_cast<const float2*>(p + (int64_t)n * D + c);
}

// ------------------------------------------------------------- sequences --

// What becomes of a sequence without tokens: its state (or the state's gradient) as it is.
__device__ __forceinline__ void pass_empty(const RecurrenceArgs& a, int n, const float* from,
                                           float* to) {
    if (to)
        for (int c = threadIdx.x & 31; c < a.D; c += 32)
            to[(int64_t)n * a.D + c] = from ? from[(int64_t)n * a.D + c] : 0.f;
}

// Finds where sequences start and end and the runs, checks the sequences and passes on the states
// of empty ones (from -> to).
__global__ void __launch_bounds__(256) setup_kernel(const RecurrenceArgs a, const Plan w,
                                                    const float* from, float* to) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    grid_dependents_launch();
    auto first = [&](int n) {
        return a.cu_seqlens ? (int64_t)__ldg(a.cu_seqlens + n) : n * (a.T_total / a.N);
    };
    // the last sequence that starts at or before token t
    auto at = [&](int64_t t) {
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first(mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    for (int64_t g = id; g * kEdge < a.T_total; g += all) {
        const int64_t t0 = g * kEdge;
        uint32_t bits = 0;
        // (of empty sequences at a token the search passes to the last; so a token takes two turns at most)
        int n = at(t0);
        for (int turn = 0; turn < 3 * kEdge && n < a.N && (bits == 0 || first(n) < t0 + kEdge);
             ++turn, ++n) {
            int64_t b, e;
            seq_range(a.cu_seqlens, n, a.N, a.T_total, nullptr, b, e);
            if (b >= e) {
                if (first(n) >= t0 + kEdge) break;
                n = max(n, at(first(n)) - 1);
                continue;
            }
            if (b >= t0 && b < t0 + kEdge) {
                bits |= 1u << (b - t0);
                w.start_seq[b] = n;
            }
            if (e > t0 && e <= t0 + kEdge) {
                bits |= 256u << (e - 1 - t0);
                w.end_seq[e - 1] = n;
            }
            if (e > t0 + kEdge - 1 || b >= t0 + kEdge) break;
        }
        w.marks[g] = bits;
    }
    // a run has the sequences that start in its part of the tokens
    for (int64_t r = id; r <= w.runs; r += all) {
        int64_t t = a.T_total * r / w.runs;
        if (r > 0 && r < w.runs) {
            const int n = at(t - 1) + 1;  // the first that starts at or after t
            t = n < a.N ? min(max(first(n), (int64_t)0), a.T_total) : a.T_total;
        }
        w.run[r] = (int)t;
    }
    for (int64_t n = id / 32; n < a.N; n += all / 32) {
        int64_t b, e;
        seq_range(a.cu_seqlens, (int)n, a.N, a.T_total,
                  (threadIdx.x & 31) == 0 ? a.dev_err : nullptr, b, e);
        if (b >= e) pass_empty(a, (int)n, from, to);
    }
}

// ------------------------------------------------------------------ scan --

// A channel's map (p, H).  p stands for P: P - 1 where that is -1/2 or more, P itself, or the next to
// nothing in place of zero, below; kConstant where the map is constant.
constexpr float kConstant = 2.f, kNothing = 1.2e-38f;
__device__ __forceinline__ bool constant(float p) { return p > 1.f; }
__device__ __forceinline__ float apply(float2 m, float h) {
    float r = m.y;
    if (!constant(m.x)) r = fmaf(m.x, h, m.y);
    if (m.x <= 0.f) r += h;
    return r;
}
// p of tokens without a cut, whose gates add up to w.
__device__ __forceinline__ float decay(float w, float near) {
    return w >= -0.6f ? near : fmaxf(ex2_approx(w * kLog2e), kNothing);
}
__device__ __forceinline__ float2 decay(float2 w) {
    const float2 near = expm1_near(w);
    return make_float2(decay(w.x, near.x), decay(w.y, near.y));
}

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// p's place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t place_in(const void* p, unsigned rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    return at;
}
// Writes v there, and counts its bytes on a barrier there.
__device__ __forceinline__ void send(uint32_t at, uint32_t done, float2 v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::
                     "r"(at), "f"(v.x), "f"(v.y), "r"(done)
                 : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------- the loop --

// Of tokens t .. t + kTok - 1: those that start a sequence, and from bit 16 those that end one.  By a
// whole warp.
template <int kTok>
__device__ __forceinline__ uint32_t marks_of(const Plan& w, const int2* few, int lane, int t,
                                             int64_t T) {
    uint32_t m = 0;
    if (few == nullptr && w.marks) {
#pragma unroll
        for (int j = 0; j < kTok; j += kEdge) {
            const uint32_t v = t + j < T ? __ldg(w.marks + (t + j) / kEdge) : 0u;
            m |= (v & 0xffu) << j | (v >> 8) << (16 + j);
        }
        return m;
    }
    if (few == nullptr) {  // one sequence
        if (t == 0) m = 1u;
        if (T > t && T <= t + kTok) m |= 0x10000u << (int)(T - 1 - t);
        return m;
    }
    const unsigned first = few[lane].x - t, last = few[lane].y - t;
    if (first < kTok) m = 1u << first;
    if (last < kTok) m |= 0x10000u << last;
    return __reduce_or_sync(~0u, m);
}

// A CTA's tiles in its cluster's run.  Step k's is the `place(k)`-th in the scan's order; there may be
// none left for this CTA.
template <bool kBwd, int kT>
struct Steps {
    int begin, end, base, tiles, count, rank, ctas;
    __device__ __forceinline__ Steps(int b, int e)
        : begin(b), end(e), base(b / kEdge * kEdge), rank((int)cluster_rank()), ctas((int)cluster_size()) {
        tiles = (end - base + kT - 1) / kT;
        count = (tiles + ctas - 1) / ctas;
    }
    __device__ __forceinline__ bool some(int k) const { return k * ctas + rank < tiles; }
    // this CTA's tiles
    __device__ __forceinline__ int own() const { return (tiles - rank + ctas - 1) / ctas; }
    // the bytes of a step's maps from the cluster
    __device__ __forceinline__ uint32_t bytes() const { return ctas * kC * (uint32_t)sizeof(float2); }
    __device__ __forceinline__ int first_token(int k) const {
        const int p = k * ctas + rank;
        return base + (kBwd ? tiles - 1 - p : p) * kT;
    }
};

// What a CTA keeps of a step's maps, in the scan's order, by channels.
template <int kStages>
struct Maps {
    float2 warps[kWarps][kC];          // its warps'
    float2 tiles[2][kMaxCluster][kC];  // the cluster's tiles'; of two steps in turn
    float start[kWarps][kC];           // the sums of its warps' gates, then the states they start from
    float carry[kC];                   // from step to step
    int2 few[kFew];                    // a few sequences' first and last tokens (kNone: empty)
    uint64_t there[2], states, full[kStages];  // barriers: the tiles', the states, inputs are there

    // a thread's two channels of them
    __device__ __forceinline__ void put(int turn, int lane, float2 p, float2 H) {
        *reinterpret_cast<float4*>(&warps[turn][2 * lane]) = make_float4(p.x, H.x, p.y, H.y);
    }
    __device__ __forceinline__ float2& states_of(int turn, int lane) {
        return *reinterpret_cast<float2*>(&start[turn][2 * lane]);
    }
};
constexpr int kCarriers = kC / 32;  // warps that exchange, a lane a channel

// By the first kCarriers warps, with the warps' maps there: sends the tile's map to the CTAs of the
// cluster, carries the state over the cluster's maps and leaves the warps' starts.  (Every warp for
// itself would read most of the maps again, some 800 instructions a step more with 8 CTAs; by one
// warp, two channels a lane, 65,536 x 4096 took 464 us instead of 449.)
template <int kStages, typename Steps>
__device__ __forceinline__ void exchange(Maps<kStages>& x, const Steps& steps, int k, int c,
                                         bool& broken, unsigned* err) {
    const int buf = k & 1;
    float H = 0.f, sum = 0.f;
    bool cut = false;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
        const float2 m = x.warps[j][c];
        H = apply(m, H);
        sum += x.start[j][c];
        cut |= constant(m.x);
    }
    const float2 all = make_float2(cut ? kConstant : decay(sum, expm1_near(both(sum)).x), H);
    for (int j = 0; j < steps.ctas; ++j)
        send(place_in(&x.tiles[buf][steps.rank][c], j), place_in(&x.there[buf], j), all);
    // (the next maps for this buffer are sent when this CTA's of the next step are there, which its
    // barrier of that step precedes)
    if (!mbar_wait(&x.there[buf], k / 2 & 1, err))
        broken = true;
    else if (c == 0)
        mbar_expect_tx(&x.there[buf], steps.bytes());
    float h = k == 0 ? 0.f : x.carry[c], mine = h;
#pragma unroll 4
    for (int j = 0; j < kMaxCluster; ++j) {
        if (j >= steps.ctas) break;
        if (j == steps.rank) mine = h;
        h = apply(x.tiles[buf][j][c], h);
    }
    x.carry[c] = h;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) {
        x.start[j][c] = mine;
        mine = apply(x.warps[j][c], mine);
    }
    __syncwarp();
    if (c % 32 == 0) mbar_arrive(&x.states);
}

// Before anything else: the barriers, by all threads; the caller waits for the cluster
// (cluster_wait) before it sends.
template <typename In, int kStages>
__device__ __forceinline__ void open_maps(Maps<kStages>& x, const Tensors& m, uint32_t bytes) {
    if (threadIdx.x == 0) {
        for (int k = 0; k < kStages; ++k) mbar_init(&x.full[k], fill_count<In>(m));
        for (int k = 0; k < 2; ++k) mbar_init(&x.there[k], 1);
        mbar_init(&x.states, kCarriers);
        fence_mbar_init();
        for (int k = 0; k < 2; ++k) mbar_expect_tx(&x.there[k], bytes);
    }
    __syncthreads();
    cluster_arrive();
}

// After the last step, by all threads, until nobody in the cluster can send here.  Where a wait ran out,
// a CTA leaves the steps at the next barrier, step k (it fills no stage and arms no barrier whose phase it
// has not seen end), and waits first for what is on its way all the same, with limits: the last fills
// of the stages, and the maps of step k, which is the last that other CTAs can send without its own.
template <int kStages, typename Steps>
__device__ __forceinline__ void close_maps(Maps<kStages>& x, const Steps& steps, int k, int ahead,
                                           bool broken, unsigned* err) {
    if (__syncthreads_or(broken)) {
        const int s = threadIdx.x;
        if (s < kStages) {
            if (const int fills = ring_fills(min(k + ahead, steps.own()), s, kStages))
                mbar_wait(&x.full[s], fills - 1 & 1, err);
        } else if (s == 32) {
            for (int j = max(k - 1, 0); j <= k && j < steps.count; ++j)
                mbar_wait(&x.there[j & 1], j / 2 & 1, err);
        }
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
}

// The cluster's run and first channel; false where it has nothing to do.  With `few` a CTA reads the
// offsets itself, a lane of every warp one sequence, and takes on what the setup launch does.
__device__ __forceinline__ bool find_run(const RecurrenceArgs& a, const Plan& w, int2* few, int lane,
                                         const float* from, float* to, int& begin, int& end,
                                         int& c0) {
    const int id = blockIdx.x / cluster_size(), r = id / w.cols;
    c0 = (id - r * w.cols) * kC;
    if (few == nullptr && w.run) {
        begin = w.run[r];
        end = w.run[r + 1];
        return begin < end;
    }
    if (few == nullptr) {
        begin = 0;
        end = (int)a.T_total;
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            int64_t b, e;
            seq_range(a.cu_seqlens, 0, 1, a.T_total, a.dev_err, b, e);
        }
        return true;
    }
    const bool mine = lane < a.N;
    int64_t b = 0, e = 0;
    if (mine)
        seq_range(a.cu_seqlens, lane, a.N, a.T_total, blockIdx.x == 0 ? a.dev_err : nullptr, b, e);
    if (threadIdx.x < 32)
        few[lane] = b < e ? make_int2((int)b, (int)e - 1) : make_int2(kNone, kNone);
    const bool passes = mine && b >= e && to && r == 0 && cluster_rank() == 0 && threadIdx.x < 32;
    for (unsigned empty = __ballot_sync(~0u, passes); empty; empty &= empty - 1) {
        const int n = __ffs(empty) - 1;
        if (c0 + 2 * lane < a.D) {
            const int64_t at = (int64_t)n * a.D + c0 + 2 * lane;
            store_pair(to + at, from ? pair(from + at) : both(0.f));
        }
    }
    // a run has the sequences that start in its part of the tokens
    auto bound = [&](int j) {
        const int t = (int)(a.T_total * j / w.runs);
        return j == 0 ? 0
               : j == w.runs
                   ? t
                   : __reduce_min_sync(~0u, b < e && b >= t ? (int)b : (int)a.T_total);
    };
    begin = bound(r);
    end = bound(r + 1);
    return begin < end;
}
// The sequence that starts, or ends, with token t.
__device__ __forceinline__ int find_few(const int* first_or_last, int t) {
    int n = 0;
    while (n < kFew - 1 && first_or_last[2 * n] != t) ++n;
    return n;
}
__device__ __forceinline__ int start_at(const Plan& w, const int2* few, int64_t t) {
    return few ? find_few(&few[0].x, (int)t) : w.start_seq ? w.start_seq[t] : 0;
}
__device__ __forceinline__ int end_at(const Plan& w, const int2* few, int64_t t) {
    return few ? find_few(&few[0].y, (int)t) : w.end_seq ? w.end_seq[t] : 0;
}

// ---------------------------------------------------------------- forward --

template <typename In, typename IO, int kTok, int kStages, bool kOnlyEdges, bool kFewOnes>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(
    const __grid_constant__ RecurrenceArgs a, const __grid_constant__ Plan w,
    const __grid_constant__ GateBound gb, const __grid_constant__ Tensors m) {
    using S = Stage<In, IO, false, kTok>;
    extern __shared__ __align__(128) char ring[];
    __shared__ Maps<kStages> x;
    grid_dependency_wait();
    int begin, end, c0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int2* const few = kFewOnes ? x.few : nullptr;
    if (!find_run(a, w, few, lane, a.h0, a.h_out, begin, end, c0)) return;
    const int ch = c0 + 2 * lane;
    const bool live = ch < a.D;
    const Steps<false, S::kT> steps(begin, end);
    open_maps<In>(x, m, steps.bytes());
    bool broken = false;  // (a wait that ran out)
    auto fill = [&](int k) {
        if (warp != kCarriers || !steps.some(k)) return;
        char* const st = ring + k % kStages * S::kBytes;
        uint64_t* const full = &x.full[k % kStages];
        Exps<S::kT> exps;
        load_stage<S, In, IO, false>(a, m, st, full, steps.first_token(k), c0, lane, exps);
        put_exps<S, In>(st, full, lane, exps);
    };
    auto marks_at = [&](int k) {
        return steps.some(k)
                   ? marks_of<kTok>(w, few, lane, steps.first_token(k) + warp * kTok, a.T_total)
                   : 0u;
    };
#pragma unroll
    for (int k = 0; k < kStages; ++k) fill(k);
    const float2 nl =
        channel_rate(live ? *reinterpret_cast<const float2*>(a.A_log + ch) : both(0.f), 0.f).neg_log2;
    __syncwarp();
    cluster_wait();
    uint32_t marks = marks_at(0);
    int k = 0;
    for (; k < steps.count; ++k) {
        const int s = k % kStages;
        const View<S, In, IO> v{ring + s * S::kBytes, nullptr, warp, lane};
        const int64_t t = steps.first_token(k) + warp * kTok;
        const bool some = steps.some(k);
        // of every token: the decay from before the warp's tokens to after it, and the state after it
        // if that before them were zero
        float2 c[kTok], nb[kTok], opening[kTok / kEdge] = {};
        float2 P = both(1.f), H = both(0.f);
        if (!some) {
            x.states_of(warp, lane) = both(0.f);
            x.put(warp, lane, both(0.f), both(0.f));  // (what leaves a state as it is)
        } else {
            if (!mbar_wait(&x.full[s], k / kStages & 1, a.dev_err)) broken = true;
            recurrence_steps([&](int which, int j) { return v.input(which, j); }, nl, gb, c, nb,
                             [&](float2 sum) {
                                 sum = mul_pair(sum, both(gb.g_min));
                                 x.states_of(warp, lane) = sum;
                             });
            if ((marks & 0xffffu) == 0u) {
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    P = fma_pair(c[j], P, P);
                    H = recurrence_next(c[j], nb[j], H);
                    c[j] = P;
                    nb[j] = H;
                }
                x.put(warp, lane, decay(x.states_of(warp, lane)), H);
            } else {
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    if (marks >> j & 1) {
                        P = both(kConstant);  // (from here on)
                        H = both(0.f);
                        if (a.h0 && live) H = state_row(a.h0, start_at(w, few, t + j), a.D, ch);
                        if (j % kEdge == 0) opening[j / kEdge] = H;
                    }
                    if (!constant(P.x)) P = fma_pair(c[j], P, P);
                    H = recurrence_next(c[j], nb[j], H);
                    c[j] = P;
                    nb[j] = H;
                }
                x.put(warp, lane, both(kConstant), H);
            }
        }
        if (__syncthreads_or(broken)) break;
        if (warp < kCarriers) exchange(x, steps, k, threadIdx.x, broken, a.dev_err);
        fill(k + kStages);  // (the stage has been read; by another warp)
        const uint32_t coming = marks_at(k + 1);
        if (!mbar_wait(&x.states, k & 1, a.dev_err)) broken = true;
        const float2 h = x.states_of(warp, lane);
        if (some && live) {
            IO* y = static_cast<IO*>(a.y) + t * a.D + ch;
            float* edge = a.edges + t / kEdge * a.D + ch;
            if (marks == 0u && t >= begin && t + kTok <= end) {
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    if (j % kEdge == 0 && a.edges)
                        store_pair(edge + j / kEdge * (int64_t)a.D,
                                   j == 0 ? h : fma_pair(c[j - 1], h, nb[j - 1]));
                    if (!kOnlyEdges) store_pair(y, fma_pair(c[j], h, nb[j]));
                    y += a.D;
                }
            } else {
                float2 last = h;
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    const bool in = t + j >= begin && t + j < end;
                    if (j % kEdge == 0 && a.edges && in)
                        store_pair(edge + j / kEdge * (int64_t)a.D,
                                   marks >> j & 1 ? opening[j / kEdge] : last);
                    last = constant(c[j].x) ? nb[j] : fma_pair(c[j], h, nb[j]);
                    if (!kOnlyEdges && in) {
                        store_pair(y, last);
                        if (marks >> (16 + j) & 1 && a.h_out)
                            store_pair(a.h_out + (int64_t)end_at(w, few, t + j) * a.D + ch, last);
                    }
                    y += a.D;
                }
            }
        }
        marks = coming;
    }
    close_maps(x, steps, k, kStages, broken, a.dev_err);
}

// -------------------------------------------------------------- gradients --

template <typename In, typename IO, int kStages>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(
    const __grid_constant__ RecurrenceArgs a, const __grid_constant__ Plan w,
    const __grid_constant__ GateBound gb, const __grid_constant__ Tensors m, float* part) {
    constexpr int kTok = kEdge;  // (a warp's states come from its edge)
    using S = Stage<In, IO, true, kTok>;
    constexpr int kAhead = kStages - 1;  // steps from the one at hand to the one loaded
    extern __shared__ __align__(128) char ring[];
    __shared__ Maps<kStages> x;
    grid_dependency_wait();
    int begin, end, c0;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool any = find_run(a, w, nullptr, lane, nullptr, nullptr, begin, end, c0);
    const int ch = c0 + 2 * lane;
    const int turn = kWarps - 1 - warp;  // in the scan's order
    const bool live = ch < a.D;
    __shared__ float2 sums[kThreads];  // dA_log, a thread's tokens so far (steps' sums are added up)
    sums[threadIdx.x] = both(0.f);
    if (any) {
        const Steps<true, S::kT> steps(begin, end);
        open_maps<In>(x, m, steps.bytes());
        bool broken = false;
        auto fill = [&](int k) {
            if (warp != kCarriers || !steps.some(k)) return;
            char* const st = ring + k % kStages * S::kBytes;
            uint64_t* const full = &x.full[k % kStages];
            Exps<S::kT> exps;
            load_stage<S, In, IO, true>(a, m, st, full, steps.first_token(k), c0, lane, exps);
            put_exps<S, In>(st, full, lane, exps);
        };
        // a step's marks, and the state that the warp's tokens start from
        auto marks_at = [&](int k) {
            return steps.some(k)
                       ? marks_of<kTok>(w, nullptr, lane, steps.first_token(k) + warp * kTok, a.T_total)
                       : 0u;
        };
        auto edge_at = [&](int k) {
            const int64_t t = steps.first_token(k) + warp * kTok;
            return steps.some(k) && t < a.T_total && live
                       ? __ldg(reinterpret_cast<const float2*>(a.edges + t / kEdge * a.D + ch))
                       : both(0.f);
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fill(k);
        const ChannelRate r = channel_rate(
            live ? *reinterpret_cast<const float2*>(a.A_log + ch) : both(0.f), gb.g_min);
        float2 edge = edge_at(0);
        __syncwarp();
        cluster_wait();
        uint32_t marks = marks_at(0);
        int k = 0;
        for (; k < steps.count; ++k) {
            const int s = k % kStages;
            char* const st = ring + s * S::kBytes;
            const View<S, In, IO> v{st, S::kInPlace ? st : ring + kStages * S::kBytes, warp, lane};
            const int t0 = steps.first_token(k);
            const int64_t t = t0 + warp * kTok;
            const bool some = steps.some(k), whole = some && t0 >= begin && t0 + S::kT <= end;
            // the negated factors of l in the gradients, from the states; the scan's state is -r, what
            // -l_t has from later tokens: r_{t-1} = a_t (dy_t + r_t)
            float2 c[kTok], fx[kTok], fz[kTok], fi[kTok];
            float2 H = both(0.f);
            if (!some) {
                x.states_of(turn, lane) = both(0.f);
                x.put(turn, lane, both(0.f), both(0.f));
            } else {
                if (!mbar_wait(&x.full[s], k / kStages & 1, a.dev_err)) broken = true;
                auto in = [&](int which, int j) { return v.input(which, j); };
                auto summed = [&](float2 sum) {
                    sum = mul_pair(sum, both(gb.g_min));
                    x.states_of(turn, lane) = sum;
                };
                if ((marks & 0xffffu) == 0u)
                    recurrence_grads(in, r, gb, edge, [](int, float2 h) { return h; }, c, fx, fz, fi, summed);
                else
                    recurrence_grads(
                        in, r, gb, edge,
                        [&](int j, float2 h) {
                            if (marks >> j & 1)
                                h = a.h0 && live ? state_row(a.h0, start_at(w, nullptr, t + j), a.D, ch)
                                                 : both(0.f);
                            return h;
                        },
                        c, fx, fz, fi, summed);
                if (marks >> 16 == 0u) {
#pragma unroll
                    for (int j = kTok - 1; j >= 0; --j) {
                        const float2 l = fma_pair(v.dy(j), both(-1.f), H);
                        H = fma_pair(c[j], l, l);
                    }
                    x.put(turn, lane, decay(x.states_of(turn, lane)), H);
                } else {
#pragma unroll
                    for (int j = kTok - 1; j >= 0; --j) {
                        if (marks >> (16 + j) & 1)
                            H = a.dh_out && live
                                    ? mul_pair(state_row(a.dh_out, end_at(w, nullptr, t + j), a.D, ch),
                                               both(-1.f))
                                    : both(0.f);
                        const float2 l = fma_pair(v.dy(j), both(-1.f), H);
                        H = fma_pair(c[j], l, l);
                    }
                    x.put(turn, lane, both(kConstant), H);
                }
            }
            if (threadIdx.x == 0) bulk_wait_read0();  // (the stage before this one is free)
            if (__syncthreads_or(broken)) break;
            if (warp < kCarriers) exchange(x, steps, k, threadIdx.x, broken, a.dev_err);
            fill(k + kAhead);  // (by another warp)
            edge = edge_at(k + 1);
            const uint32_t coming = marks_at(k + 1);
            if (!mbar_wait(&x.states, k & 1, a.dev_err)) broken = true;
            float2 nr = x.states_of(turn, lane), dA = both(0.f);
            // a token's gradients but for the state's
            auto take = [&](int j, float2 l, IO* dx, IO* dz, IO* di) {
                const float2 g = mul_pair(l, fz[j]), z = v.finite(1, j);
                store_pair(dx, mul_pair(l, fx[j]));
                store_pair(dz, g);
                store_pair(di, mul_pair(l, fi[j]));
                dA = fma_pair(g, z, dA);
            };
            if (whole && marks == 0u) {
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) {
                    const float2 l = fma_pair(v.dy(j), both(-1.f), nr);
                    nr = fma_pair(c[j], l, l);
                    take(j, l, v.out(0, j), v.out(1, j), v.out(2, j));
                }
            } else if (some) {
                const int64_t at = t * a.D + ch;
#pragma unroll
                for (int j = kTok - 1; j >= 0; --j) {
                    if (marks >> (16 + j) & 1)
                        nr = a.dh_out && live
                                 ? mul_pair(state_row(a.dh_out, end_at(w, nullptr, t + j), a.D, ch),
                                            both(-1.f))
                                 : both(0.f);
                    const float2 l = fma_pair(v.dy(j), both(-1.f), nr);
                    nr = fma_pair(c[j], l, l);
                    const bool mine_too = live && t + j >= begin && t + j < end;
                    const int64_t o = at + (int64_t)j * a.D;
                    if (whole)
                        take(j, l, v.out(0, j), v.out(1, j), v.out(2, j));
                    else if (mine_too)
                        take(j, l, static_cast<IO*>(a.dx) + o, static_cast<IO*>(a.dz) + o,
                             static_cast<IO*>(a.di) + o);
                    if (mine_too && marks >> j & 1 && a.dh0)
                        store_pair(a.dh0 + (int64_t)start_at(w, nullptr, t + j) * a.D + ch,
                                   mul_pair(nr, both(-1.f)));
                }
            }
            sums[threadIdx.x] = add_pair(sums[threadIdx.x], dA);
            if (whole) {  // the tile's results leave when all warps' are there
                fence_async_smem();
                if (warp > 0) {
                    asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
                } else {
                    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
                    if (lane == 0) {
#pragma unroll
                        for (int o = 0; o < 3; ++o) tma_store(&m.out[o], v.outs + o * S::kOut, c0, t0);
                        bulk_commit();
                    }
                    __syncwarp();
                }
            }
            marks = coming;
        }
        if (threadIdx.x == 0) bulk_wait0();
        close_maps(x, steps, k, kAhead, broken, a.dev_err);
    }
    if (part == nullptr) return;
    // the CTA's dA_log: over the warps, in a fixed order
    __syncthreads();
    if (threadIdx.x < 32 && live) {
        float2 s = sums[lane];
#pragma unroll
        for (int j = 1; j < kWarps; ++j) s = add_pair(s, sums[j * 32 + lane]);
        const unsigned ctas = cluster_size();
        const int64_t row = (int64_t)(blockIdx.x / ctas / w.cols) * ctas + cluster_rank();
        *reinterpret_cast<float2*>(part + row * a.D + ch) = s;
    }
}

// dA_log[c] = the sum of the CTAs' parts in a fixed order: a CTA takes 32 channels, its 32 warps every
// 32nd part (4 us, latency).
__global__ void __launch_bounds__(1024) rate_kernel(const float* part, int parts, int D, float* dA) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    grid_dependency_wait();
    float x = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int b = warp; b < parts; b += 32) x += part[(int64_t)b * D + c];
    }
    red[warp][lane] = x;
    __syncthreads();
    if (warp == 0 && c < D) {
        x = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) x += red[j][lane];
        dA[c] = x;
    }
}

// ------------------------------------------------------- the single token --

// Four channels a thread; bound by memory, or by its launch: 256 requests x 4096 3.4 us, 4.9 TB/s with
// the states in the second-level cache, of a call of 14.
__device__ __forceinline__ float4 four(const __nv_bfloat16* p) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float4 four(const float* p) {
    return __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ void store_four(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store_four(float* p, float4 v) {
    *reinterpret_cast<float4*>(p) = v;
}

template <typename IO>
__global__ void __launch_bounds__(128) step_kernel(const IO* x, int64_t x_ld, const IO* z,
                                                   int64_t z_ld, const IO* i, int64_t i_ld,
                                                   const float* A_log, GateBound gb, float* h,
                                                   const int32_t* slots, int n_slots, int64_t N,
                                                   int D, IO* y, unsigned* err) {
    const int64_t id = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int per_row = D / 4;
    const int64_t n = id / per_row;
    const int c = (int)(id - n * per_row) * 4;
    if (n >= N) return;
    int64_t slot = slots ? __ldg(slots + n) : n;
    const float4 xv = four(x + n * x_ld + c), zv = four(z + n * z_ld + c),
                 iv = four(i + n * i_ld + c);
    const float4 A = __ldg(reinterpret_cast<const float4*>(A_log + c));
    if (slot >= n_slots) {
        if (c == 0) atomicOr(err, kDevErrBadSlot);
        slot = -1;
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (slot >= 0) {
        float4* hp = reinterpret_cast<float4*>(h + slot * D + c);
        v = *hp;
        const float2 in[3][2] = {{make_float2(xv.x, xv.y), make_float2(xv.z, xv.w)},
                                 {make_float2(zv.x, zv.y), make_float2(zv.z, zv.w)},
                                 {make_float2(iv.x, iv.y), make_float2(iv.z, iv.w)}};
        auto next = [&](int j, float2 Ae, float2 he) {
            float2 cc[1], nb[1];
            recurrence_steps([&](int which, int) { return in[which][j]; },
                             channel_rate(Ae, 0.f).neg_log2, gb, cc, nb, [](float2) {});
            return recurrence_next(cc[0], nb[0], he);
        };
        const float2 a = next(0, make_float2(A.x, A.y), make_float2(v.x, v.y));
        const float2 b = next(1, make_float2(A.z, A.w), make_float2(v.z, v.w));
        v = make_float4(a.x, a.y, b.x, b.y);
        *hp = v;
    }
    store_four(y + n * D + c, v);
}

// --------------------------------------------------------------- launches --

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// Runs are as many as sequences, but of 1,024 tokens on average at least, and 8 times what the GPU
// holds at most.
int count_runs(int64_t T, int N, int cols) {
    const int64_t most = std::max<int64_t>(1, 152 * 2 * 8 / cols);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(N, T / 1024), most));
}

// CTAs of a cluster, for tiles of kT tokens: as many as keep all of them on the GPU at once, counted as
// two an SM (the gradients into fp32 have one there at a time); with several runs, one for every 1,024
// tokens that a run has on average.  (That number comes from 24 sequences, 47,139 tokens x 2560: 186 us
// with two, 197 with one, 199 with four.  Batches much unlike it were not tuned for.)
int count_ctas(int64_t T, int runs, int cols, int kT) {
    int n = 1;
    while (2 * n <= kMaxCluster && T > (int64_t)kT * n * runs &&
           ((int64_t)runs * cols * 2 * n <= 304 || (runs > 1 && T >= (int64_t)1024 * n * runs)))
        n *= 2;
    return n;
}

// Whether the forward's CTAs find their way through the sequences by themselves, without the setup
// launch and its workspace: where a call's latency counts more than the scan's, which this makes 10 to
// 20 % longer.  Calls without and with a setup launch: 252 tokens x 1024 in 4 sequences 21 and 28 us,
// 2,048 x 1024 21 and 27, 512 x 4096 in 32 20 and 27, but 8,192 x 1024 in 24 26 either way (as graphs
// 26 and 22) and 8,192 x 2560 69 and 60.  (The gradients have no registers left for it.)
bool few_ones(int64_t T, int N, int cols) {
    return T > 0 && N > 1 && N <= kFew && T * cols <= 65536;
}

// The parts of a workspace; w may be nullptr.
size_t lay_out(char* ws, int64_t T, int N, int D, bool bwd, Plan* w, float** edges, float** part) {
    size_t n = 0;
    auto take = [&](size_t bytes) {
        char* p = ws ? ws + n : nullptr;
        n += up(bytes);
        return p;
    };
    Plan s{};
    s.cols = (D + kC - 1) / kC;
    s.runs = count_runs(T, N, s.cols);
    s.few = !bwd && few_ones(T, N, s.cols);
    if ((N > 1 && !s.few) || T == 0) {  // (a setup launch; without tokens it passes the states on)
        s.run = reinterpret_cast<int*>(take((s.runs + 1) * 4));
        s.marks = reinterpret_cast<uint32_t*>(take((T + kEdge - 1) / kEdge * 4));
        s.start_seq = reinterpret_cast<int*>(take(T * 4));
        s.end_seq = reinterpret_cast<int*>(take(T * 4));
    }
    if (bwd) {
        char* p = take((size_t)s.runs * kMaxCluster * D * 4);
        char* e = take((size_t)((T + kEdge - 1) / kEdge) * D * 4);
        if (part) *part = reinterpret_cast<float*>(p);
        if (edges) *edges = reinterpret_cast<float*>(e);
    }
    if (w) *w = s;
    return n;
}

cudaError_t setup(const RecurrenceArgs& a, const Plan& w, const float* from, float* to) {
    if (w.run == nullptr) return cudaSuccess;
    const int64_t want = std::max<int64_t>(a.T_total / kEdge, (int64_t)a.N * 32);
    const int grid = (int)std::min<int64_t>(want / 256 + 1, 152 * 8);
    ProfScope prof("recurrence_setup_kernel", a.stream);
    setup_kernel<<<grid, 256, 0, a.stream>>>(a, w, from, to);
    return cudaGetLastError();
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// [T][D] of E with a token stride of ld elements.
template <typename E>
bool make_map(CUtensorMap* m, const void* base, int64_t T, int D, int64_t ld, int kT) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)T};
    const cuuint64_t stride = (cuuint64_t)ld * sizeof(E);
    const cuuint32_t box[2] = {kC, (cuuint32_t)kT}, estr[2] = {1, 1};
    return fn(m,
              sizeof(E) == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
              : sizeof(E) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
              2, const_cast<void*>(base), dims, &stride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename S, typename In, typename IO>
bool make_maps(Tensors& m, const RecurrenceArgs& a, bool bwd) {
    const int64_t T = a.T_total;
    auto of = [&](auto* type, int which, const void* base, int64_t ld, bool out) {
        using E = std::remove_pointer_t<decltype(type)>;
        return make_map<E>(out ? &m.out[which] : &m.in[which], base, T, a.D, ld, S::kT);
    };
    In* in = nullptr;
    IO* io = nullptr;
    m.plain = sizeof(In) == 1 && a.D % 16 != 0;
    if (!m.plain && !(of(in, 0, a.x, a.x_ld, false) && of(in, 1, a.z, a.z_ld, false) &&
                      of(in, 2, a.i, a.i_ld, false)))
        return false;
    if (!bwd) return true;
    return (m.plain || of(io, 3, a.dy, a.dy_ld, false)) && of(io, 0, a.dx, a.D, true) &&
           of(io, 1, a.dz, a.D, true) && of(io, 2, a.di, a.D, true);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_scan(void (*kernel)(KArgs...), const char* name, int smem, int ctas,
                        const RecurrenceArgs& a, const Plan& w, Args... args) {
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
        return e;
    ProfScope prof(name, a.stream);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)w.runs * w.cols * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, w, gate_bound(a.g_min), args...);
}

// A warp's tokens in the forward: 16 of them halve what the steps cost beside the tokens' arithmetic;
// 8 of fp32, whose tiles would leave one CTA an SM.  (Of the gradients' type where only edges are
// wanted, so that these are the same for packed inputs and the values they stand for.)
template <typename IO>
constexpr int kForwardTok = sizeof(IO) == 4 ? 8 : 16;

template <typename In, typename IO, bool kOnlyEdges>
cudaError_t forward(const RecurrenceArgs& a, const Plan& w) {
    constexpr int kTok = kForwardTok<IO>, kStages = 2;
    using S = Stage<In, IO, false, kTok>;
    Tensors m{};
    if (!make_maps<S, In, IO>(m, a, false)) return cudaErrorInvalidValue;
    const int ctas = count_ctas(a.T_total, w.runs, w.cols, S::kT);
    auto kernel = scan_kernel<In, IO, kTok, kStages, kOnlyEdges, false>;
    if constexpr (!kOnlyEdges)
        if (w.few) kernel = scan_kernel<In, IO, kTok, kStages, false, true>;
    return launch_scan(kernel, "recurrence_kernel", kStages * S::kBytes, ctas, a, w, m);
}

template <typename In, typename IO>
cudaError_t backward(RecurrenceArgs a) {
    constexpr int kStages = 3;
    using S = Stage<In, IO, true, kEdge>;
    Plan w;
    float *edges, *part;
    lay_out(static_cast<char*>(a.workspace), a.T_total, a.N, a.D, true, &w, &edges, &part);
    if (cudaError_t e = setup(a, w, a.dh_out, a.dh0)) return e;
    const int ctas = count_ctas(a.T_total, w.runs, w.cols, S::kT);
    if (a.T_total > 0) {
        if (a.edges == nullptr) {
            RecurrenceArgs f = a;
            f.edges = a.edges = edges;
            f.y = nullptr;
            f.h_out = nullptr;
            if (cudaError_t e = forward<In, IO, true>(f, w)) return e;
        }
        Tensors m{};
        if (!make_maps<S, In, IO>(m, a, true)) return cudaErrorInvalidValue;
        if (cudaError_t e = launch_scan(scan_bwd_kernel<In, IO, kStages>, "recurrence_bwd_kernel",
                                        kStages * S::kBytes + S::kOuts, ctas, a, w, m,
                                        a.dA_log ? part : nullptr))
            return e;
    }
    if (a.dA_log) {
        ProfScope prof("recurrence_rate_kernel", a.stream);
        return launch_dependent(rate_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, a.stream,
                                (const float*)part, a.T_total > 0 ? w.runs * ctas : 0, a.D, a.dA_log);
    }
    return cudaGetLastError();
}

template <typename IO>
cudaError_t forward_of(const RecurrenceArgs& a) {
    Plan w;
    lay_out(static_cast<char*>(a.workspace), a.T_total, a.N, a.D, false, &w, nullptr, nullptr);
    if (cudaError_t e = setup(a, w, a.h0, a.h_out)) return e;
    return a.T_total == 0 ? cudaSuccess : forward<IO, IO, false>(a, w);
}

}  // namespace

size_t recurrence_fwd_workspace_size(int64_t T, int N, int D) {
    return lay_out(nullptr, T, N, D, false, nullptr, nullptr, nullptr);
}
size_t recurrence_bwd_workspace_size(int64_t T, int N, int D) {
    return lay_out(nullptr, T, N, D, true, nullptr, nullptr, nullptr);
}

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a) {
    return a.io_bf16 ? forward_of<__nv_bfloat16>(a) : forward_of<float>(a);
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
    const int64_t grid = ((int64_t)N * (D / 4) + 127) / 128;
    ProfScope prof("recurrence_step_kernel", stream);
    auto run = [&](auto* as) {
        using T = std::remove_pointer_t<decltype(as)>;
        step_kernel<T><<<(unsigned)grid, 128, 0, stream>>>(
            static_cast<const T*>(x), x_ld, static_cast<const T*>(z), z_ld,
            static_cast<const T*>(i), i_ld, A_log, gate_bound(g_min), h, slots, n_slots, (int64_t)N, D,
            static_cast<T*>(y), dev_err);
    };
    if (io_bf16) run((__nv_bfloat16*)nullptr);
    else run((float*)nullptr);
    return cudaGetLastError();
}

}  // namespace kda
