// recurrence.cu -- the gated recurrence of single channels (declared in include/kda.h): packed
// forward, gradients (from whole or 8-bit inputs) and the single-token step.
//
//   h_t = a_t h_{t-1} + b_t,   a = e^g, b = sqrt(1 - e^{2g}) s(i) x          (recurrence_math.cuh)
//   l_t = dy_t + a_{t+1} l_{t+1}, backwards, for the gradients
//
// Both are scans of affine maps (P, H): h -> P h + H, and both run in one pass over the data.  A tile
// is 64 channels x 64 tokens: a warp holds 8 tokens, a lane two channels.  The warps compose their
// tokens' maps, one warp composes the tile's, publishes it and looks back for the state the tile
// starts from: the nearest tile before it whose end state is published, from which it applies the
// published maps in between.  Whatever it finds, the state is the same fused multiply-adds in the
// same order, P_j (... P_0 h + H_0 ...) + H_j, so results do not depend on timing.  Then every warp
// goes over its tokens again, in registers, and writes.
//   A CTA takes tiles by tickets, the columns of one row of tiles after the other, so a tile waits
// only for tiles that running CTAs have begun (however many CTAs are resident), and loads the next
// tiles' inputs (cp.async) while it waits.  A tile in which a sequence starts ends in a state that
// depends on nothing before it: its end state is published at once.
//
// The gradients go over the tiles backwards.  A warp's states come from the edges, the state that
// every 8th token starts from, which the forward writes on request; without them a forward that
// writes nothing else runs first.  So the factors of l_t in the gradients are formed once, before
// the scan, and stay in registers until l_t is known.
//
// Sequences: every tile has the sequences that touch it (a setup launch finds them, which also
// clears the flags); where one starts, the map is constant (selected, not multiplied by zero, so
// that nothing that is not finite crosses).
#include <algorithm>

#include "kda_internal.h"
#include "recurrence_math.cuh"
#include "tc_util.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kTok = 8;            // tokens a warp holds
constexpr int kWarps = 8;
constexpr int kT = kTok * kWarps;  // tokens of a tile
constexpr int kC = 64;             // channels of a tile, and of an exponent of packed inputs
constexpr int kEdge = kTok;        // tokens from one edge to the next
constexpr int kThreads = 32 * kWarps;

// What the CTAs of a launch share, in the workspace.
struct Shared {
    uint32_t* counter;  // tickets; next to it the abort flag of waits that ran out
    int2* seqs;         // [tiles] first and last sequence that may start or end in the tile, {0, -1}
                        // where none does; nullptr: one row of tiles, every sequence may
    uint32_t* flag;     // [rows][cols] 0, 1: map published, 2: end state published
    float4* map;        // [rows][cols][32] (P, H) of a lane's two channels
    float2* state;      // [rows][cols][32]
    float* part;        // [tiles][D] dA_log of the tiles
    int tiles, cols;
};

// ---------------------------------------------------------------- inputs --

// A stage of the ring: the inputs of a tile.
template <typename In, typename IO, bool kBwd>
struct Stage {
    static constexpr int kIn = kT * kC * (int)sizeof(In);
    static constexpr int kDy = 3 * kIn;
    static constexpr int kEdges = kDy + (kBwd ? kT * kC * (int)sizeof(IO) : 0);
    static constexpr int kExps = kEdges + (kBwd ? kWarps * kC * 4 : 0);
    static constexpr int kSeqs = kExps + (sizeof(In) == 1 ? 3 * kT : 0);
    static constexpr int kBytes = kSeqs + 16;
    static_assert(kIn % 16 == 0 && kDy % 16 == 0 && kEdges % 16 == 0 && kBytes % 16 == 0, "");
};

template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool live) {
    const int n = live ? kBytes : 0;
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                     "r"(n));
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src),
                     "r"(n));
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;"); }
template <int n>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// 64 tokens x 64 channels of a tensor; rows and channels past its end become zeros.
template <typename In>
__device__ __forceinline__ void load_tile(char* dst, const void* src, int64_t ld, int64_t t0, int c0,
                                          int64_t T, int D) {
    // (rows of codes begin on 8 bytes only)
    constexpr int kPiece = sizeof(In) == 1 ? 8 : 16, kElems = kPiece / (int)sizeof(In);
    constexpr int kPer = kC / kElems;
#pragma unroll
    for (int k = 0; k < kT * kPer / kThreads; ++k) {
        const int p = k * kThreads + threadIdx.x, row = p / kPer, c = p % kPer * kElems;
        const bool live = t0 + row < T && c0 + c < D;
        const In* s = static_cast<const In*>(src) + (live ? (t0 + row) * ld + c0 + c : 0);
        copy_async<kPiece>(dst + (row * kC + c) * (int)sizeof(In), s, live);
    }
}

// Starts the loads of a tile.  Of packed inputs, the exponent that this thread has to put into the
// stage (put_exps) is returned.
template <typename In, typename IO, bool kBwd>
__device__ __forceinline__ int load_stage(const RecurrenceArgs& a, const Shared& w, char* st,
                                          int tile, int col) {
    using S = Stage<In, IO, kBwd>;
    const int64_t t0 = (int64_t)tile * kT;
    const int c0 = col * kC;
    load_tile<In>(st, a.x, a.x_ld, t0, c0, a.T_total, a.D);
    load_tile<In>(st + S::kIn, a.z, a.z_ld, t0, c0, a.T_total, a.D);
    load_tile<In>(st + 2 * S::kIn, a.i, a.i_ld, t0, c0, a.T_total, a.D);
    if (kBwd) {
        load_tile<IO>(st + S::kDy, a.dy, a.dy_ld, t0, c0, a.T_total, a.D);
        if (threadIdx.x < kWarps * kC / 4) {
            const int row = threadIdx.x / (kC / 4), c = threadIdx.x % (kC / 4) * 4;
            const bool live = t0 + row * kEdge < a.T_total && c0 + c < a.D;
            copy_async<16>(st + S::kEdges + (row * kC + c) * 4,
                           a.edges + (live ? (t0 / kEdge + row) * a.D + c0 + c : 0), live);
        }
    }
    if (w.seqs && threadIdx.x == kThreads - 1) copy_async<8>(st + S::kSeqs, w.seqs + tile, true);
    if (sizeof(In) == 1 && threadIdx.x < 3 * kT) {
        const int k = threadIdx.x / kT, row = threadIdx.x % kT;
        const int8_t* e = k == 0 ? a.x_exps : k == 1 ? a.z_exps : a.i_exps;
        if (t0 + row < a.T_total) return __ldg(e + (int64_t)col * a.T_total + t0 + row);
    }
    return 0;
}
template <typename In, typename IO, bool kBwd>
__device__ __forceinline__ void put_exps(char* st, int e) {
    if (sizeof(In) == 1 && threadIdx.x < 3 * kT)
        reinterpret_cast<int8_t*>(st)[Stage<In, IO, kBwd>::kExps + threadIdx.x] = (int8_t)e;
}

__device__ __forceinline__ float2 pair(const __nv_bfloat16* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair(const float* p) {
    return *reinterpret_cast<const float2*>(p);
}

// The values of token `row` and the lane's channels of input k (x, z, i) of a stage.
template <typename In, typename IO, bool kBwd>
__device__ __forceinline__ float2 input(const char* st, int k, int row, int lane) {
    using S = Stage<In, IO, kBwd>;
    const In* p = reinterpret_cast<const In*>(st + k * S::kIn) + row * kC + 2 * lane;
    if constexpr (sizeof(In) == 1) {
        const char2 q = *reinterpret_cast<const char2*>(p);
        const int e = reinterpret_cast<const int8_t*>(st)[S::kExps + k * kT + row];
        // 2^e, denormal at -127; -128 stands for NaN
        const float s = __int_as_float(e > -127 ? (e + 127) << 23 : e == -127 ? 1 << 22 : 0x7fc00000);
        return make_float2((float)(signed char)q.x * s, (float)(signed char)q.y * s);
    } else {
        return pair(p);
    }
}

__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void store_pair(float* p, float2 v) {
    *reinterpret_cast<float2*>(p) = v;
}

// ------------------------------------------------------------- sequences --

// Where sequences start and end in a tile.
struct Marks {
    unsigned long long starts, ends;  // bits of the tile's tokens
    int start_seq[kT], end_seq[kT];   // valid where the bit is set
};

// Marks the sequences lo .. hi; called by all threads.
__device__ __forceinline__ void mark(const RecurrenceArgs& a, Marks& m, int64_t t0, int lo, int hi) {
    if (threadIdx.x == 0) m.starts = m.ends = 0ull;
    __syncthreads();
    for (int n = lo + threadIdx.x; n <= hi; n += kThreads) {
        int64_t b, e;
        seq_range(a.cu_seqlens, n, a.N, a.T_total, nullptr, b, e);
        if (b >= e) continue;
        if (b >= t0 && b < t0 + kT) {
            m.start_seq[b - t0] = n;
            atomicOr(&m.starts, 1ull << (b - t0));
        }
        if (e > t0 && e <= t0 + kT) {
            m.end_seq[e - 1 - t0] = n;
            atomicOr(&m.ends, 1ull << (e - 1 - t0));
        }
    }
    __syncthreads();
}

// What becomes of a sequence without tokens: its state (or the state's gradient) as it is.
__device__ __forceinline__ void pass_empty(const RecurrenceArgs& a, int n, int c, const float* from,
                                           float* to) {
    if (to) to[(int64_t)n * a.D + c] = from ? from[(int64_t)n * a.D + c] : 0.f;
}

// Clears what the scan's CTAs share, finds the sequences of every tile, checks the sequences and
// passes on the states of empty ones (from -> to).
__global__ void __launch_bounds__(256) setup_kernel(const RecurrenceArgs a, const Shared w,
                                                    const float* from, float* to) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    grid_dependents_launch();
    if (id < 2) w.counter[id] = 0u;
    for (int64_t k = id; k < (int64_t)w.tiles * w.cols; k += all) w.flag[k] = 0u;
    // the last sequence that starts at or before token t
    auto at = [&](int64_t t) {
        if (a.cu_seqlens == nullptr) return (int)min(t / (a.T_total / a.N), (int64_t)a.N - 1);
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(a.cu_seqlens + mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    for (int64_t k = id; k < w.tiles; k += all) {
        const int64_t t0 = k * kT, t1 = min(t0 + kT, a.T_total);
        const int lo = at(t0), hi = at(t1 - 1);
        int64_t b, e;
        seq_range(a.cu_seqlens, lo, a.N, a.T_total, nullptr, b, e);
        w.seqs[k] = lo == hi && b != t0 && e > t1 ? make_int2(0, -1) : make_int2(lo, hi);
    }
    const int lane = threadIdx.x & 31;
    for (int64_t n = id / 32; n < a.N; n += all / 32) {
        int64_t b, e;
        seq_range(a.cu_seqlens, (int)n, a.N, a.T_total, lane == 0 ? a.dev_err : nullptr, b, e);
        if (b >= e)
            for (int c = lane; c < a.D; c += 32) pass_empty(a, (int)n, c, from, to);
    }
}

// ------------------------------------------------------------- look back --

// The state before row p of a column (rows in the scan's order); called by a whole warp, a lane for
// its two channels.
__device__ __forceinline__ float2 look_back(const Shared& w, int p, int col, int lane,
                                            unsigned* err) {
    int first;
    uint64_t since = 0;
    for (int spins = 0;; ++spins) {
        const int q = p - 1 - lane;
        // (before the first row: a state of zero)
        const uint32_t f = q >= 0 ? ld_acquire_gpu(w.flag + (int64_t)q * w.cols + col) : 2u;
        const unsigned ended = __ballot_sync(0xffffffffu, f == 2u);
        const unsigned known = __ballot_sync(0xffffffffu, f != 0u);
        first = __ffs(ended) - 1;
        if (ended && (~known & ((1u << first) - 1u)) == 0u) break;
        if (spins < 16) continue;
        int stop = 0;
        if (lane == 0) {
            const uint64_t now = globaltimer();
            if (since == 0) since = now;
            stop = *reinterpret_cast<volatile uint32_t*>(w.counter + 1) != 0u;
            if (!stop && now - since > kWaitLimitNs) {
                atomicOr(err, kDevErrTimeout);
                atomicExch(w.counter + 1, 1u);
                stop = 1;
            }
        }
        if (__shfl_sync(0xffffffffu, stop, 0)) return make_float2(0.f, 0.f);
    }
    __syncwarp();
    int q = p - 1 - first;
    float2 h = make_float2(0.f, 0.f);
    if (q >= 0) h = __ldcg(w.state + ((int64_t)q * w.cols + col) * 32 + lane);
    const float4* m = w.map + (int64_t)col * 32 + lane;
    const int64_t step = (int64_t)w.cols * 32;
    for (++q; q < p; q += 8) {
        float4 g[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (q + k < p) g[k] = __ldcg(m + (q + k) * step);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (q + k < p) h = make_float2(fmaf(g[k].x, h.x, g[k].y), fmaf(g[k].z, h.y, g[k].w));
    }
    return h;
}

__device__ __forceinline__ void publish_map(const Shared& w, int p, int col, int lane, float4 m) {
    const int64_t at = (int64_t)p * w.cols + col;
    __stcg(w.map + at * 32 + lane, m);
    __syncwarp();
    if (lane == 0) st_release_gpu(w.flag + at, 1u);
}
__device__ __forceinline__ void publish_state(const Shared& w, int p, int col, int lane, float2 h) {
    const int64_t at = (int64_t)p * w.cols + col;
    __stcg(w.state + at * 32 + lane, h);
    __syncwarp();
    if (lane == 0) st_release_gpu(w.flag + at, 2u);
}

// The warps' maps of a tile, and the state that it starts from.
struct Compose {
    float4 map[kWarps][32];
    float2 in[32];
};

// Called by one warp with all maps there: the tile's map (cut: a bit for every warp whose map is
// constant, in the scan's order), its publication, and the state the tile starts from.
__device__ __forceinline__ void compose(const Shared& w, Compose& s, unsigned cut, bool fresh, int p,
                                        int col, int lane, unsigned* err) {
    if (w.seqs == nullptr) {  // one row of tiles: a state of zero, and none that waits for this one
        s.in[lane] = make_float2(0.f, 0.f);
        return;
    }
    float4 m = s.map[0][lane];
#pragma unroll
    for (int j = 1; j < kWarps; ++j) {
        const float4 g = s.map[j][lane];
        if (cut >> j & 1)
            m = g;
        else
            m = make_float4(m.x * g.x, fmaf(g.x, m.y, g.y), m.z * g.z, fmaf(g.z, m.w, g.w));
    }
    const bool last = p == w.tiles - 1;  // nobody waits for it
    if (!last) {
        if (cut) publish_state(w, p, col, lane, make_float2(m.y, m.w));
        else publish_map(w, p, col, lane, m);
    }
    float2 h = make_float2(0.f, 0.f);
    if (!fresh) {  // (a sequence that starts with the tile takes nothing in)
        h = look_back(w, p, col, lane, err);
        if (!cut && !last)
            publish_state(w, p, col, lane, make_float2(fmaf(m.x, h.x, m.y), fmaf(m.z, h.y, m.w)));
    }
    s.in[lane] = h;
}

// The state that warp `warp` (in the scan's order) starts from.
__device__ __forceinline__ float2 warp_state(const Compose& s, unsigned cut, int warp, int lane) {
    float2 h = s.in[lane];
#pragma unroll
    for (int j = 0; j < kWarps - 1; ++j) {
        if (j < warp) {
            const float4 g = s.map[j][lane];
            h = cut >> j & 1 ? make_float2(g.y, g.w)
                             : make_float2(fmaf(g.x, h.x, g.y), fmaf(g.z, h.y, g.w));
        }
    }
    return h;
}

// A bit for every group of 8 tokens of which one is marked.
__device__ __forceinline__ unsigned groups_of(unsigned long long marks) {
    unsigned g = 0;
#pragma unroll
    for (int j = 0; j < kWarps; ++j) g |= (marks >> (kTok * j) & 0xffull) ? 1u << j : 0u;
    return g;
}

// ------------------------------------------------------------- the loops --

// Runs body(stage, tile, col) over a CTA's tiles, their inputs loaded ahead.
template <typename In, typename IO, bool kBwd, int kStages, typename Body>
__device__ __forceinline__ void for_tiles(const RecurrenceArgs& a, const Shared& w, char* ring,
                                          Body&& body) {
    using S = Stage<In, IO, kBwd>;
    __shared__ uint32_t ticket[kStages];  // of the tile in each stage
    const uint32_t all = (uint32_t)w.tiles * (uint32_t)w.cols;
    auto load = [&](int s) {
        int e = 0;
        const uint32_t id = ticket[s];
        if (id < all) {
            const int p = id / w.cols, tile = kBwd ? w.tiles - 1 - p : p;
            e = load_stage<In, IO, kBwd>(a, w, ring + s * S::kBytes, tile, id % w.cols);
        }
        copy_commit();
        return e;
    };
    if (threadIdx.x == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s)
            ticket[s] = w.seqs ? atomicAdd(w.counter, 1u) : s == 0 ? blockIdx.x : all;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) put_exps<In, IO, kBwd>(ring + s * S::kBytes, load(s));
    for (int s = 0;;) {
        copy_wait<kStages - 2>();
        __syncthreads();  // the stage is there, and the one before it free
        const uint32_t id = ticket[s];
        if (id >= all) break;
        const int free = s == 0 ? kStages - 1 : s - 1;
        const int e = load(free);
        uint32_t next = all;  // (on its way while this tile is worked on)
        if (threadIdx.x == 0 && w.seqs) next = atomicAdd(w.counter, 1u);
        const int p = id / w.cols, col = id % w.cols;
        body(ring + s * S::kBytes, p, kBwd ? w.tiles - 1 - p : p, col);
        put_exps<In, IO, kBwd>(ring + free * S::kBytes, e);
        // (every thread has read this stage's ticket before the body's barriers)
        if (threadIdx.x == 0) ticket[s] = next;
        s = s + 1 == kStages ? 0 : s + 1;
    }
    copy_wait<0>();
}

template <typename In, typename IO, bool kBwd>
__device__ __forceinline__ void find_marks(const RecurrenceArgs& a, const Shared& w, const char* st,
                                           int tile, Marks& marks, unsigned long long& starts,
                                           unsigned long long& ends) {
    starts = ends = 0ull;
    const int2 q = w.seqs ? *reinterpret_cast<const int2*>(st + Stage<In, IO, kBwd>::kSeqs)
                          : make_int2(0, a.N - 1);
    if (q.x > q.y) return;
    mark(a, marks, (int64_t)tile * kT, q.x, q.y);
    starts = marks.starts;
    ends = marks.ends;
}

// ---------------------------------------------------------------- forward --

template <typename In, typename IO, int kStages, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) scan_kernel(
    const __grid_constant__ RecurrenceArgs a, const __grid_constant__ Shared w) {
    extern __shared__ __align__(128) char ring[];
    __shared__ Compose comp;
    __shared__ Marks marks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_dependents_launch();
    if (w.seqs == nullptr) {  // no setup launch: its checks here
        const int c = blockIdx.x * kC + 2 * lane;
        for (int n = warp; n < a.N; n += kWarps) {
            int64_t b, e;
            seq_range(a.cu_seqlens, n, a.N, a.T_total, lane == 0 ? a.dev_err : nullptr, b, e);
            if (b >= e && c < a.D) {
                pass_empty(a, n, c, a.h0, a.h_out);
                pass_empty(a, n, c + 1, a.h0, a.h_out);
            }
        }
    }
    for_tiles<In, IO, false, kStages>(a, w, ring, [&](const char* st, int p, int tile, int col) {
        const int64_t t0 = (int64_t)tile * kT;
        const int c0 = col * kC + 2 * lane;
        const bool live = c0 < a.D;
        unsigned long long starts, ends;
        find_marks<In, IO, false>(a, w, st, tile, marks, starts, ends);
        const unsigned my_starts = starts >> (kTok * warp) & 0xffu;
        const unsigned my_ends = ends >> (kTok * warp) & 0xffu;
        const float2 A = live ? *reinterpret_cast<const float2*>(a.A_log + c0) : make_float2(0.f, 0.f);
        const float nx = channel_rate(A.x).neg_log2, ny = channel_rate(A.y).neg_log2;

        float2 c[kTok], b[kTok];
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const int row = warp * kTok + k;
            const float2 x = input<In, IO, false>(st, 0, row, lane);
            const float2 z = input<In, IO, false>(st, 1, row, lane);
            const float2 i = input<In, IO, false>(st, 2, row, lane);
            const Step u = recurrence_step(x.x, z.x, i.x, nx, a.g_min);
            const Step v = recurrence_step(x.y, z.y, i.y, ny, a.g_min);
            c[k] = make_float2(u.c, v.c);
            b[k] = make_float2(u.b, v.b);
        }
        float2 first = make_float2(0.f, 0.f);  // the initial state of a sequence that starts here
        if (my_starts && a.h0) {  // initial states: into the first tokens' input terms
            float2 h0[kTok];
#pragma unroll
            for (int k = 0; k < kTok; ++k)
                h0[k] = my_starts >> k & 1 && live
                            ? *reinterpret_cast<const float2*>(
                                  a.h0 + (int64_t)marks.start_seq[warp * kTok + k] * a.D + c0)
                            : make_float2(0.f, 0.f);
            first = h0[0];
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                b[k].x = recurrence_next(c[k].x, b[k].x, h0[k].x);
                b[k].y = recurrence_next(c[k].y, b[k].y, h0[k].y);
            }
        }
        float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            if (my_starts >> k & 1) m = make_float4(0.f, 0.f, 0.f, 0.f);
            m.x = fmaf(c[k].x, m.x, m.x);
            m.z = fmaf(c[k].y, m.z, m.z);
            m.y = recurrence_next(c[k].x, b[k].x, m.y);
            m.w = recurrence_next(c[k].y, b[k].y, m.w);
        }
        comp.map[warp][lane] = m;
        __syncthreads();
        const unsigned cut = groups_of(starts);
        if (warp == 0) compose(w, comp, cut, starts & 1ull, p, col, lane, a.dev_err);
        __syncthreads();
        float2 h = warp_state(comp, cut, warp, lane);
        const int64_t t = t0 + warp * kTok;
        if (a.edges && live && t < a.T_total)
            *reinterpret_cast<float2*>(a.edges + (t / kEdge) * a.D + c0) = my_starts & 1 ? first : h;
        IO* y = static_cast<IO*>(a.y) + t * a.D + c0;
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            if (my_starts >> k & 1) h = make_float2(0.f, 0.f);
            h.x = recurrence_next(c[k].x, b[k].x, h.x);
            h.y = recurrence_next(c[k].y, b[k].y, h.y);
            if (live && t + k < a.T_total) {
                if (a.y) store_pair(y + (int64_t)k * a.D, h);
                if (my_ends >> k & 1 && a.h_out)
                    store_pair(a.h_out + (int64_t)marks.end_seq[warp * kTok + k] * a.D + c0, h);
            }
        }
    });
}

// -------------------------------------------------------------- gradients --

template <typename In, typename IO, int kStages, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) scan_bwd_kernel(
    const __grid_constant__ RecurrenceArgs a, const __grid_constant__ Shared w) {
    extern __shared__ __align__(128) char ring[];
    __shared__ Compose comp;
    __shared__ Marks marks;
    __shared__ float2 sums[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_dependents_launch();
    if (w.seqs == nullptr) {
        const int c = blockIdx.x * kC + 2 * lane;
        for (int n = warp; n < a.N; n += kWarps) {
            int64_t b, e;
            seq_range(a.cu_seqlens, n, a.N, a.T_total, lane == 0 ? a.dev_err : nullptr, b, e);
            if (b >= e && c < a.D) {
                pass_empty(a, n, c, a.dh_out, a.dh0);
                pass_empty(a, n, c + 1, a.dh_out, a.dh0);
            }
        }
    }
    for_tiles<In, IO, true, kStages>(a, w, ring, [&](const char* st, int p, int tile, int col) {
        using S = Stage<In, IO, true>;
        const int64_t t0 = (int64_t)tile * kT;
        const int c0 = col * kC + 2 * lane;
        const bool live = c0 < a.D;
        unsigned long long starts, ends;
        find_marks<In, IO, true>(a, w, st, tile, marks, starts, ends);
        const unsigned my_starts = starts >> (kTok * warp) & 0xffu;
        const unsigned my_ends = ends >> (kTok * warp) & 0xffu;
        const float2 A = live ? *reinterpret_cast<const float2*>(a.A_log + c0) : make_float2(0.f, 0.f);
        const ChannelRate rx = channel_rate(A.x), ry = channel_rate(A.y);

        // the factors of l in the gradients, from the states
        float2 c[kTok], fx[kTok], fz[kTok], fi[kTok], dy[kTok];
        float2 h = *reinterpret_cast<const float2*>(st + S::kEdges + (warp * kC + 2 * lane) * 4);
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const int row = warp * kTok + k;
            if (my_starts >> k & 1)
                h = a.h0 && live ? *reinterpret_cast<const float2*>(
                                       a.h0 + (int64_t)marks.start_seq[row] * a.D + c0)
                                 : make_float2(0.f, 0.f);
            const float2 x = input<In, IO, true>(st, 0, row, lane);
            const float2 z = input<In, IO, true>(st, 1, row, lane);
            const float2 i = input<In, IO, true>(st, 2, row, lane);
            const StepGrad u = recurrence_grad(x.x, z.x, i.x, rx.rate, rx.neg_log2, a.g_min, h.x);
            const StepGrad v = recurrence_grad(x.y, z.y, i.y, ry.rate, ry.neg_log2, a.g_min, h.y);
            c[k] = make_float2(u.c, v.c);
            fx[k] = make_float2(u.dx, v.dx);
            fz[k] = make_float2(u.dz, v.dz);
            fi[k] = make_float2(u.di, v.di);
            h.x = recurrence_next(u.c, u.dx * x.x, h.x);
            h.y = recurrence_next(v.c, v.dx * x.y, h.y);
            dy[k] = pair(reinterpret_cast<const IO*>(st + S::kDy) + row * kC + 2 * lane);
        }
        if (my_ends && a.dh_out) {
            float2 d[kTok];
#pragma unroll
            for (int k = 0; k < kTok; ++k)
                d[k] = my_ends >> k & 1 && live
                           ? *reinterpret_cast<const float2*>(
                                 a.dh_out + (int64_t)marks.end_seq[warp * kTok + k] * a.D + c0)
                           : make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                dy[k].x += d[k].x;
                dy[k].y += d[k].y;
            }
        }
        // r, what l_t has from later tokens: r_{t-1} = a_t (dy_t + r_t)
        float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            if (my_ends >> k & 1) m = make_float4(0.f, 0.f, 0.f, 0.f);
            m.x = fmaf(c[k].x, m.x, m.x);
            m.z = fmaf(c[k].y, m.z, m.z);
            const float lx = dy[k].x + m.y, ly = dy[k].y + m.w;
            m.y = fmaf(c[k].x, lx, lx);
            m.w = fmaf(c[k].y, ly, ly);
        }
        const int turn = kWarps - 1 - warp;  // the warp's place in the scan
        comp.map[turn][lane] = m;
        __syncthreads();
        const unsigned cut = __brev(groups_of(ends)) >> (32 - kWarps);
        if (warp == 0)
            compose(w, comp, cut, ends >> (kT - 1) & 1ull, p, col, lane, a.dev_err);
        __syncthreads();
        float2 r = warp_state(comp, cut, turn, lane);
        const int64_t t = t0 + warp * kTok;
        const int64_t at = t * a.D + c0;
        float2 dA = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            if (my_ends >> k & 1) r = make_float2(0.f, 0.f);
            const float2 l = make_float2(dy[k].x + r.x, dy[k].y + r.y);
            r.x = fmaf(c[k].x, l.x, l.x);
            r.y = fmaf(c[k].y, l.y, l.y);
            if (live && t + k < a.T_total) {
                const int64_t o = at + (int64_t)k * a.D;
                const float2 dz = make_float2(l.x * fz[k].x, l.y * fz[k].y);
                store_pair(static_cast<IO*>(a.dx) + o, make_float2(l.x * fx[k].x, l.y * fx[k].y));
                store_pair(static_cast<IO*>(a.dz) + o, dz);
                store_pair(static_cast<IO*>(a.di) + o, make_float2(l.x * fi[k].x, l.y * fi[k].y));
                // (an infinite z has a gradient of zero)
                const float2 z = input<In, IO, true>(st, 1, warp * kTok + k, lane);
                dA.x += dz.x == 0.f ? 0.f : dz.x * z.x;
                dA.y += dz.y == 0.f ? 0.f : dz.y * z.y;
                if (my_starts >> k & 1 && a.dh0)
                    store_pair(a.dh0 + (int64_t)marks.start_seq[warp * kTok + k] * a.D + c0, r);
            }
        }
        if (a.dA_log) {
            sums[warp][lane] = dA;
            __syncthreads();
            if (warp == 0 && live) {
                float2 s = sums[0][lane];
#pragma unroll
                for (int j = 1; j < kWarps; ++j) {
                    s.x += sums[j][lane].x;
                    s.y += sums[j][lane].y;
                }
                *reinterpret_cast<float2*>(w.part + (int64_t)tile * a.D + c0) = s;
            }
        }
    });
}

// dA_log[c] = the sum of the tiles' parts in a fixed order: a CTA takes 32 channels, its 32 warps
// every 32nd tile.
__global__ void __launch_bounds__(1024) rate_kernel(const float* part, int tiles, int D, float* dA) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    grid_dependency_wait();
    float x = 0.f;
    if (c < D) {
#pragma unroll 4
        for (int b = warp; b < tiles; b += 32) x += part[(int64_t)b * D + c];
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

// Four channels a thread.
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
                                                   const float* A_log, float g_min, float* h,
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
        auto next = [&](float xe, float ze, float ie, float Ae, float he) {
            const Step s = recurrence_step(xe, ze, ie, channel_rate(Ae).neg_log2, g_min);
            return recurrence_next(s.c, s.b, he);
        };
        v = make_float4(next(xv.x, zv.x, iv.x, A.x, v.x), next(xv.y, zv.y, iv.y, A.y, v.y),
                        next(xv.z, zv.z, iv.z, A.z, v.z), next(xv.w, zv.w, iv.w, A.w, v.w));
        *hp = v;
    }
    store_four(y + n * D + c, v);
}

// --------------------------------------------------------------- launches --

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// The parts of a workspace for T tokens; w may be nullptr.
size_t lay_out(char* ws, int64_t T, int D, bool bwd, Shared* w, float** edges) {
    const size_t tiles = (size_t)((T + kT - 1) / kT), cols = (D + kC - 1) / kC;
    size_t n = 0;
    auto take = [&](size_t bytes) {
        char* p = ws ? ws + n : nullptr;
        n += up(bytes);
        return p;
    };
    Shared s{};
    s.tiles = (int)tiles;
    s.cols = (int)cols;
    if (tiles != 1) {
        s.counter = reinterpret_cast<uint32_t*>(take(8));
        s.seqs = reinterpret_cast<int2*>(take(tiles * sizeof(int2)));
        s.flag = reinterpret_cast<uint32_t*>(take(tiles * cols * 4));
        s.map = reinterpret_cast<float4*>(take(tiles * cols * 32 * sizeof(float4)));
        s.state = reinterpret_cast<float2*>(take(tiles * cols * 32 * sizeof(float2)));
    }
    if (bwd) {
        s.part = reinterpret_cast<float*>(take(tiles * D * 4));
        char* e = take((size_t)((T + kEdge - 1) / kEdge) * D * 4);
        if (edges) *edges = reinterpret_cast<float*>(e);
    }
    if (w) *w = s;
    return n;
}

template <typename Kernel>
cudaError_t launch_scan(Kernel kernel, const char* name, int smem, int ctas, const RecurrenceArgs& a,
                        const Shared& w, const float* from, float* to) {
    if (w.tiles != 1) {
        const int64_t want = std::max<int64_t>((int64_t)w.tiles * w.cols / 4, (int64_t)a.N * 32);
        const int grid = (int)std::min<int64_t>((want + 255) / 256, 152 * 8);
        ProfScope prof("recurrence_setup_kernel", a.stream);
        setup_kernel<<<std::max(grid, 1), 256, 0, a.stream>>>(a, w, from, to);
    }
    if (w.tiles == 0) return cudaGetLastError();
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
        return e;
    // (one row of tiles: a CTA a column, no tickets)
    const int64_t all = (int64_t)w.tiles * w.cols;
    const int64_t grid = w.tiles == 1 ? all : std::min<int64_t>(all, 152 * ctas);
    ProfScope prof(name, a.stream);
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), smem, a.stream, a, w);
}

template <typename In, typename IO>
cudaError_t forward(const RecurrenceArgs& a, const Shared& w) {
    constexpr int kStages = 2, kCtas = sizeof(In) == 4 ? 2 : 3;
    constexpr int kSmem = kStages * Stage<In, IO, false>::kBytes;
    return launch_scan(scan_kernel<In, IO, kStages, kCtas>, "recurrence_kernel", kSmem, kCtas, a, w,
                       a.h0, a.h_out);
}

template <typename In, typename IO>
cudaError_t backward(RecurrenceArgs a) {
    Shared w;
    float* edges;
    lay_out(static_cast<char*>(a.workspace), a.T_total, a.D, true, &w, &edges);
    if (a.edges == nullptr) {
        RecurrenceArgs f = a;
        f.edges = a.edges = edges;
        f.y = nullptr;
        f.h_out = nullptr;
        if (cudaError_t e = forward<In, IO>(f, w)) return e;
    }
    constexpr int kStages = sizeof(In) == 4 ? 2 : 3, kCtas = sizeof(In) == 4 ? 1 : 2;
    constexpr int kSmem = kStages * Stage<In, IO, true>::kBytes;
    if (cudaError_t e = launch_scan(scan_bwd_kernel<In, IO, kStages, kCtas>, "recurrence_bwd_kernel",
                                    kSmem, kCtas, a, w, a.dh_out, a.dh0))
        return e;
    if (a.dA_log) {
        ProfScope prof("recurrence_rate_kernel", a.stream);
        return launch_dependent(rate_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, a.stream,
                                (const float*)w.part, w.tiles, a.D, a.dA_log);
    }
    return cudaGetLastError();
}

}  // namespace

size_t recurrence_fwd_workspace_size(int64_t T, int, int D) {
    return lay_out(nullptr, T, D, false, nullptr, nullptr);
}
size_t recurrence_bwd_workspace_size(int64_t T, int, int D) {
    return lay_out(nullptr, T, D, true, nullptr, nullptr);
}

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a) {
    Shared w;
    lay_out(static_cast<char*>(a.workspace), a.T_total, a.D, false, &w, nullptr);
    return a.io_bf16 ? forward<__nv_bfloat16, __nv_bfloat16>(a, w) : forward<float, float>(a, w);
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
            static_cast<const T*>(i), i_ld, A_log, g_min, h, slots, n_slots, (int64_t)N, D,
            static_cast<T*>(y), dev_err);
    };
    if (io_bf16) run((__nv_bfloat16*)nullptr);
    else run((float*)nullptr);
    return cudaGetLastError();
}

}  // namespace kda
