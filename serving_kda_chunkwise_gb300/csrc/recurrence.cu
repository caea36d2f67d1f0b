// recurrence.cu -- the gated recurrence of single channels (declared in include/kda.h): packed
// forward, gradients (from whole or 8-bit inputs) and the single-token step.
//
//   h_t = a_t h_{t-1} + b_t,   a = e^g, b = sqrt(1 - e^{2g}) s(i) x          (recurrence_math.cuh)
//   l_t = dy_t + a_{t+1} l_{t+1}, backwards, for the gradients
//
// Both are scans of affine maps (P, H): h -> P h + H, and both run in one pass over the data.  A tile
// is 64 channels x 64 or 128 tokens: a warp holds 8 or 16 tokens, a lane two channels.  The warps
// compose their tokens' maps, one warp composes the tile's, publishes it and looks back for the
// state the tile starts from: the nearest tile before it whose end state is published, from which
// it applies the published maps in between.  Whatever it finds, the state is the same fused
// multiply-adds in the same order, P_j (... P_0 h + H_0 ...) + H_j, so results do not depend on
// timing.  Then every warp goes over its tokens again, in registers, and writes.
//   A map or state is published as 64-bit messages, a channel's (P, H) with P's sign bit (P >= 0) or
// (state, 1), which are read whole or not at all: to wait for one is to read it until it is there,
// without a flag of its own to be read before it.
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
// clears the messages); where one starts, the map is constant (selected, not multiplied by zero, so
// that nothing that is not finite crosses).
#include <algorithm>

#include "kda_internal.h"
#include "recurrence_math.cuh"
#include "tc_util.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kWarps = 8;
constexpr int kC = 64;    // channels of a tile, and of an exponent of packed inputs
constexpr int kEdge = 8;  // tokens from one edge to the next
constexpr int kThreads = 32 * kWarps;

// What the CTAs of a launch share, in the workspace.
struct Shared {
    uint32_t* counter;  // tickets; next to it the abort flag of waits that ran out
    int2* seqs;         // [rows] first and last sequence that may start or end in the tiles of a row,
                        // {0, -1} where none does; nullptr: one row, every sequence may
    ulonglong2* mail;   // [rows][cols][map, state][32] messages of a lane's two channels
    float* part;        // [rows][D] dA_log of the tiles
    int rows, cols;
};

// ---------------------------------------------------------------- inputs --

// A stage of the ring: the inputs of a tile.
template <typename In, typename IO, bool kBwd, int kTok>
struct Stage {
    static constexpr int kT = kTok * kWarps;  // tokens of a tile
    static constexpr int kIn = kT * kC * (int)sizeof(In);
    static constexpr int kDy = 3 * kIn;
    static constexpr int kEdges = kDy + (kBwd ? kT * kC * (int)sizeof(IO) : 0);
    static constexpr int kExps = kEdges + (kBwd ? kT / kEdge * kC * 4 : 0);
    static constexpr int kSeqs = kExps + (sizeof(In) == 1 ? 3 * kT : 0);
    static constexpr int kBytes = kSeqs + 16;
    static constexpr int kExpsEach = (3 * kT + kThreads - 1) / kThreads;  // a thread's
    static_assert(kIn % 16 == 0 && kDy % 16 == 0 && kEdges % 16 == 0 && kBytes % 16 == 0, "");
    static_assert(!kBwd || kTok == kEdge, "a warp's states come from its edge");
};

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool live) {
    const int n = live ? kBytes : 0;
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n));
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n));
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;"); }
template <int n>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// kT tokens x 64 channels of a tensor; rows and channels past its end become zeros.
template <typename In, int kT>
__device__ __forceinline__ void load_tile(char* dst, const void* src, int64_t ld, int64_t t0, int c0,
                                          int64_t T, int D) {
    // (rows of codes begin on 8 bytes only)
    constexpr int kPiece = sizeof(In) == 1 ? 8 : 16, kElems = kPiece / (int)sizeof(In);
    constexpr int kPer = kC / kElems, kRows = kThreads / kPer;
    const int row = threadIdx.x / kPer, c = threadIdx.x % kPer * kElems;
    const int left = (int)min((int64_t)kT, T - t0) - row;  // rows left from this thread's first
    const bool in = c0 + c < D;
    const In* s = static_cast<const In*>(src) + (t0 + row) * ld + c0 + c;
    uint32_t d = smem_u32(dst) + (row * kC + c) * (int)sizeof(In);
#pragma unroll
    for (int k = 0; k < kT / kRows; ++k) {
        const bool live = in && k * kRows < left;
        copy_async<kPiece>(d, live ? s : src, live);
        s += kRows * ld;
        d += kRows * kC * (int)sizeof(In);
    }
}

// The exponents of packed inputs that a thread has to put into a stage.
template <int n>
struct Exps {
    int8_t e[n];
};

// Starts the loads of a tile.
template <typename S, typename In, typename IO, bool kBwd>
__device__ __forceinline__ void load_stage(const RecurrenceArgs& a, const Shared& w, char* st,
                                           int row, int col, Exps<S::kExpsEach>& exps) {
    const int64_t t0 = (int64_t)row * S::kT;
    const int c0 = col * kC;
    load_tile<In, S::kT>(st, a.x, a.x_ld, t0, c0, a.T_total, a.D);
    load_tile<In, S::kT>(st + S::kIn, a.z, a.z_ld, t0, c0, a.T_total, a.D);
    load_tile<In, S::kT>(st + 2 * S::kIn, a.i, a.i_ld, t0, c0, a.T_total, a.D);
    if (kBwd) {
        load_tile<IO, S::kT>(st + S::kDy, a.dy, a.dy_ld, t0, c0, a.T_total, a.D);
        if (threadIdx.x < S::kT / kEdge * kC / 4) {
            const int e = threadIdx.x / (kC / 4), c = threadIdx.x % (kC / 4) * 4;
            const bool live = t0 + e * kEdge < a.T_total && c0 + c < a.D;
            copy_async<16>(smem_u32(st + S::kEdges) + (e * kC + c) * 4,
                           a.edges + (live ? (t0 / kEdge + e) * a.D + c0 + c : 0), live);
        }
    }
    if (w.seqs && threadIdx.x == kThreads - 1)
        copy_async<8>(smem_u32(st + S::kSeqs), w.seqs + row, true);
    if (sizeof(In) == 1) {
#pragma unroll
        for (int j = 0; j < S::kExpsEach; ++j) {
            const int n = j * kThreads + threadIdx.x, k = n / S::kT, t = n % S::kT;
            const int8_t* e = k == 0 ? a.x_exps : k == 1 ? a.z_exps : a.i_exps;
            exps.e[j] = 0;
            if (n < 3 * S::kT && t0 + t < a.T_total)
                exps.e[j] = __ldg(e + (int64_t)col * a.T_total + t0 + t);
        }
    }
}
template <typename S, typename In>
__device__ __forceinline__ void put_exps(char* st, const Exps<S::kExpsEach>& exps) {
    if (sizeof(In) == 1) {
#pragma unroll
        for (int j = 0; j < S::kExpsEach; ++j)
            if (j * kThreads + threadIdx.x < 3 * S::kT)
                reinterpret_cast<int8_t*>(st)[S::kExps + j * kThreads + threadIdx.x] = exps.e[j];
    }
}

__device__ __forceinline__ float2 pair(const __nv_bfloat16* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair(const float* p) {
    return *reinterpret_cast<const float2*>(p);
}

// The values of token t of the tile and the lane's channels of input k (x, z, i) of a stage.
template <typename S, typename In>
__device__ __forceinline__ float2 input(const char* st, int k, int t, int lane) {
    const In* p = reinterpret_cast<const In*>(st + k * S::kIn) + t * kC + 2 * lane;
    if constexpr (sizeof(In) == 1) {
        const char2 q = *reinterpret_cast<const char2*>(p);
        const int e = reinterpret_cast<const int8_t*>(st)[S::kExps + k * S::kT + t];
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
// The lane's channels of row n of an fp32 [N, D] tensor.
__device__ __forceinline__ float2 state_row(const float* p, int n, int D, int c0) {
    return *reinterpret_cast<const float2*>(p + (int64_t)n * D + c0);
}

// ------------------------------------------------------------- sequences --

// Where sequences start and end in a tile: bits of a warp's tokens, and of the warps that have one.
template <int kT>
struct Marks {
    unsigned starts[kWarps], ends[kWarps], start_warps, end_warps;
    int start_seq[kT], end_seq[kT];  // valid where the token's bit is set
};

// Marks the sequences lo .. hi; called by all threads.
template <int kT>
__device__ __forceinline__ void mark(const RecurrenceArgs& a, Marks<kT>& m, int64_t t0, int lo,
                                     int hi) {
    constexpr int kTok = kT / kWarps;
    if (threadIdx.x < kWarps) m.starts[threadIdx.x] = m.ends[threadIdx.x] = 0u;
    if (threadIdx.x == 0) m.start_warps = m.end_warps = 0u;
    __syncthreads();
    for (int n = lo + threadIdx.x; n <= hi; n += kThreads) {
        int64_t b, e;
        seq_range(a.cu_seqlens, n, a.N, a.T_total, nullptr, b, e);
        if (b >= e) continue;
        if (b >= t0 && b < t0 + kT) {
            const int t = (int)(b - t0);
            m.start_seq[t] = n;
            atomicOr(&m.starts[t / kTok], 1u << t % kTok);
            atomicOr(&m.start_warps, 1u << t / kTok);
        }
        if (e > t0 && e <= t0 + kT) {
            const int t = (int)(e - 1 - t0);
            m.end_seq[t] = n;
            atomicOr(&m.ends[t / kTok], 1u << t % kTok);
            atomicOr(&m.end_warps, 1u << t / kTok);
        }
    }
    __syncthreads();
}

// What becomes of a sequence without tokens: its state (or the state's gradient) as it is.
__device__ __forceinline__ void pass_empty(const RecurrenceArgs& a, int n, int c, const float* from,
                                           float* to) {
    if (to) to[(int64_t)n * a.D + c] = from ? from[(int64_t)n * a.D + c] : 0.f;
}

// Checks the sequences and passes on the states of empty ones (from -> to), for a column of
// channels; called by all threads where there is no setup launch.
__device__ __forceinline__ void check_sequences(const RecurrenceArgs& a, int c, const float* from,
                                                float* to) {
    for (int n = threadIdx.x >> 5; n < a.N; n += kWarps) {
        int64_t b, e;
        seq_range(a.cu_seqlens, n, a.N, a.T_total, (threadIdx.x & 31) == 0 ? a.dev_err : nullptr, b,
                  e);
        if (b >= e && c < a.D) {
            pass_empty(a, n, c, from, to);
            pass_empty(a, n, c + 1, from, to);
        }
    }
}

// Clears what the scan's CTAs share, finds the sequences of every row of tiles, checks the sequences
// and passes on the states of empty ones (from -> to).
__global__ void __launch_bounds__(256) setup_kernel(const RecurrenceArgs a, const Shared w, int kT,
                                                    const float* from, float* to) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    grid_dependents_launch();
    if (id < 2) w.counter[id] = 0u;
    for (int64_t k = id; k < (int64_t)w.rows * w.cols * 64; k += all)
        w.mail[k] = make_ulonglong2(0ull, 0ull);
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
    for (int64_t k = id; k < w.rows; k += all) {
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

// ------------------------------------------------------------- messages --

__device__ __forceinline__ ulonglong2 read_mail(const ulonglong2* p) {
    ulonglong2 v;
    asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];"
                 : "=l"(v.x), "=l"(v.y)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void send_mail(ulonglong2* p, ulonglong2 v) {
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(v.x), "l"(v.y)
                 : "memory");
}
__device__ __forceinline__ unsigned long long message(uint32_t lo, float hi) {
    return (unsigned long long)__float_as_uint(hi) << 32 | lo;
}
__device__ __forceinline__ float high(unsigned long long m) {
    return __uint_as_float((uint32_t)(m >> 32));
}
__device__ __forceinline__ float factor(unsigned long long m) {
    return __uint_as_float((uint32_t)m & 0x7fffffffu);
}

// A lane's maps (P, H) of its two channels.
__device__ __forceinline__ void send_map(ulonglong2* at, float2 P, float2 H) {
    send_mail(at, make_ulonglong2(message(__float_as_uint(P.x) | 0x80000000u, H.x),
                                  message(__float_as_uint(P.y) | 0x80000000u, H.y)));
}
__device__ __forceinline__ void send_state(ulonglong2* at, float2 h) {
    send_mail(at + 32, make_ulonglong2(message(1u, h.x), message(1u, h.y)));
}
__device__ __forceinline__ bool has_map(ulonglong2 m) {
    return ((uint32_t)m.x & (uint32_t)m.y & 0x80000000u) != 0u;
}
__device__ __forceinline__ bool has_state(ulonglong2 m) {
    return ((uint32_t)m.x & (uint32_t)m.y & 1u) != 0u;
}
__device__ __forceinline__ float2 apply(ulonglong2 m, float2 h) {
    return make_float2(fmaf(factor(m.x), h.x, high(m.x)), fmaf(factor(m.y), h.y, high(m.y)));
}

// Bounds a wait of a whole warp: true once it has to be given up.
struct Patience {
    uint64_t since = 0;
    int spins = 0;
    __device__ __forceinline__ bool over(const Shared& w, unsigned* err, int lane) {
        if (++spins < 16) return false;
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
        return __shfl_sync(0xffffffffu, stop, 0) != 0;
    }
};

// The state before row p of a column (rows in the scan's order); called by a whole warp, a lane for
// its two channels.
__device__ __forceinline__ float2 look_back(const Shared& w, int p, int col, int lane, unsigned* err) {
    const int64_t step = (int64_t)w.cols * 64;
    const ulonglong2* at = w.mail + ((int64_t)(p - 1) * w.cols + col) * 64 + lane;  // row p - 1
    Patience wait;
    constexpr int kNear = 4;
    for (;;) {
        if (wait.over(w, err, lane)) return make_float2(0.f, 0.f);
        // the nearest rows, maps and states at once: one round trip once they are there
        ulonglong2 m[kNear], s[kNear];
#pragma unroll
        for (int k = 0; k < kNear; ++k) {
            if (k >= p) continue;
            m[k] = read_mail(at - k * step);
            s[k] = read_mail(at - k * step + 32);
        }
        int from = -1;       // rows back to a state
        bool maps = true;    // all maps on the way are there
#pragma unroll
        for (int k = 0; k < kNear; ++k) {
            if (from >= 0) continue;
            if (k >= p || has_state(s[k])) from = k;
            else maps = maps && has_map(m[k]);
        }
        float2 h = make_float2(0.f, 0.f);
        if (__all_sync(0xffffffffu, from >= 0 && maps)) {
#pragma unroll
            for (int k = kNear - 1; k >= 0; --k) {
                if (k == from && k < p) h = make_float2(high(s[k].x), high(s[k].y));
                if (k < from && k < p) h = apply(m[k], h);
            }
            return h;
        }
        if (!__all_sync(0xffffffffu, from < 0 && maps)) continue;
        // farther: the nearest state of the 32 rows before, then the maps from there
        const int q = p - 1 - lane;
        const bool some =
            q < 0 || has_state(read_mail(w.mail + ((int64_t)q * w.cols + col) * 64 + 32));
        const unsigned v = __ballot_sync(0xffffffffu, some);
        if (v == 0u) continue;
        int k = min(__ffs(v) - 1, p);
        if (k < p) {
            const ulonglong2 t = read_mail(at - k * step + 32);
            if (!__all_sync(0xffffffffu, has_state(t))) continue;
            h = make_float2(high(t.x), high(t.y));
        }
        for (--k; k >= 0;) {
            ulonglong2 g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j <= k) g[j] = read_mail(at - (k - j) * step);
            int taken = 0;
            bool go = true;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j > k) continue;
                go = go && __all_sync(0xffffffffu, has_map(g[j]));
                if (go) {
                    h = apply(g[j], h);
                    ++taken;
                }
            }
            k -= taken;
            if (!go) break;
        }
        // (a row whose map has not come may come with its state alone: from the start)
        if (k < 0) return h;
    }
}

// The warps' maps of a tile (P, H of a lane's two channels), and the state that it starts from.
struct Compose {
    float4 map[kWarps][32];
    float2 in[32];
};

// Called by one warp with all maps there: the tile's map (cut: a bit for every warp whose map is
// constant, in the scan's order), its publication, and the state the tile starts from (zero for a
// fresh one, with whose first token a sequence starts).
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
            m = make_float4(m.x * g.x, m.y * g.y, fmaf(g.x, m.z, g.z), fmaf(g.y, m.w, g.w));
    }
    ulonglong2* at = w.mail + ((int64_t)p * w.cols + col) * 64 + lane;
    const bool last = p == w.rows - 1;  // nobody waits for it
    if (!last) {
        if (cut) send_state(at, make_float2(m.z, m.w));
        else if (p > 0) send_map(at, make_float2(m.x, m.y), make_float2(m.z, m.w));
    }
    float2 h = make_float2(0.f, 0.f);
    if (!fresh) {
        h = look_back(w, p, col, lane, err);
        if (!cut && !last)
            send_state(at, make_float2(fmaf(m.x, h.x, m.z), fmaf(m.y, h.y, m.w)));
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
            h = cut >> j & 1 ? make_float2(g.z, g.w)
                             : make_float2(fmaf(g.x, h.x, g.z), fmaf(g.y, h.y, g.w));
        }
    }
    return h;
}

// ------------------------------------------------------------- the loops --

// Runs body(stage, p, row, col) over a CTA's tiles (p: the row in the scan's order), their inputs
// loaded ahead.
template <typename S, typename In, typename IO, bool kBwd, int kStages, typename Body>
__device__ __forceinline__ void for_tiles(const RecurrenceArgs& a, const Shared& w, char* ring,
                                          Body&& body) {
    __shared__ int2 tile[kStages];  // (p, column) of the tile in each stage; p = rows: none left
    auto place = [&](uint32_t id) {
        const uint32_t p = id / (uint32_t)w.cols;
        return make_int2((int)min(p, (uint32_t)w.rows), (int)(id - p * (uint32_t)w.cols));
    };
    auto load = [&](int s, Exps<S::kExpsEach>& e) {
        const int2 t = tile[s];
        if (t.x < w.rows)
            load_stage<S, In, IO, kBwd>(a, w, ring + s * S::kBytes, kBwd ? w.rows - 1 - t.x : t.x, t.y,
                                        e);
        copy_commit();
    };
    const uint32_t none = 0xffffffffu;
    if (threadIdx.x == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s)
            tile[s] = w.seqs ? place(atomicAdd(w.counter, 1u))
                             : s == 0 ? make_int2(0, blockIdx.x) : make_int2(w.rows, 0);
    }
    __syncthreads();
    Exps<S::kExpsEach> exps;
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        load(s, exps);
        put_exps<S, In>(ring + s * S::kBytes, exps);
    }
    for (int s = 0;;) {
        copy_wait<kStages - 2>();
        __syncthreads();  // the stage is there, and the one before it free
        const int2 t = tile[s];
        if (t.x >= w.rows) break;
        const int free = s == 0 ? kStages - 1 : s - 1;
        load(free, exps);
        uint32_t next = none;  // (on its way while this tile is worked on)
        if (threadIdx.x == 0 && w.seqs) next = atomicAdd(w.counter, 1u);
        body(ring + s * S::kBytes, t.x, kBwd ? w.rows - 1 - t.x : t.x, t.y);
        put_exps<S, In>(ring + free * S::kBytes, exps);
        // (every thread has read this stage's place before the body's barriers)
        if (threadIdx.x == 0) tile[s] = next == none ? make_int2(w.rows, 0) : place(next);
        s = s + 1 == kStages ? 0 : s + 1;
    }
    copy_wait<0>();
}

// Marks a tile's sequences, if any may start or end there.
template <typename S>
__device__ __forceinline__ bool find_marks(const RecurrenceArgs& a, const Shared& w, const char* st,
                                           int row, Marks<S::kT>& marks) {
    const int2 q = w.seqs ? *reinterpret_cast<const int2*>(st + S::kSeqs) : make_int2(0, a.N - 1);
    if (q.x > q.y) return false;
    mark<S::kT>(a, marks, (int64_t)row * S::kT, q.x, q.y);
    return true;
}

// ---------------------------------------------------------------- forward --

template <typename In, typename IO, int kTok, int kStages, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) scan_kernel(
    const __grid_constant__ RecurrenceArgs a, const __grid_constant__ Shared w,
    const __grid_constant__ GateBound gb) {
    using S = Stage<In, IO, false, kTok>;
    extern __shared__ __align__(128) char ring[];
    __shared__ Compose comp;
    __shared__ Marks<S::kT> marks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_dependents_launch();
    if (w.seqs == nullptr) check_sequences(a, blockIdx.x * kC + 2 * lane, a.h0, a.h_out);
    for_tiles<S, In, IO, false, kStages>(a, w, ring, [&](const char* st, int p, int row, int col) {
        const int64_t t0 = (int64_t)row * S::kT;
        const int c0 = col * kC + 2 * lane;
        const bool live = c0 < a.D;
        unsigned starts = 0, ends = 0, cut = 0;
        bool fresh = false;
        if (find_marks<S>(a, w, st, row, marks)) {
            starts = marks.starts[warp];
            ends = marks.ends[warp];
            cut = marks.start_warps;
            fresh = marks.starts[0] & 1;
        }
        const float2 nl =
            channel_rate(live ? *reinterpret_cast<const float2*>(a.A_log + c0) : both(0.f), 0.f)
                .neg_log2;

        float2 c[kTok], nb[kTok];
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const int t = warp * kTok + k;
            const Step u = recurrence_step(input<S, In>(st, 0, t, lane), input<S, In>(st, 1, t, lane),
                                           input<S, In>(st, 2, t, lane), nl, gb);
            c[k] = u.c;
            nb[k] = u.nb;
            if (k % 2 == 1) asm volatile("" ::: "memory");  // (later tokens' loads would take registers)
        }
        if (starts && a.h0) {  // initial states: into the first tokens' input terms
#pragma unroll
            for (int k = 0; k < kTok; k += 4) {
                float2 h0[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h0[j] = starts >> (k + j) & 1 && live
                                ? state_row(a.h0, marks.start_seq[warp * kTok + k + j], a.D, c0)
                                : both(0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (starts >> (k + j) & 1)
                        nb[k + j] = mul2(recurrence_next(c[k + j], nb[k + j], h0[j]), both(-1.f));
            }
        }
        float2 P = both(1.f), H = both(0.f);
        if (starts == 0) {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                P = fma2(c[k], P, P);
                H = recurrence_next(c[k], nb[k], H);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                if (starts >> k & 1) H = both(0.f);
                H = recurrence_next(c[k], nb[k], H);
            }
        }
        comp.map[warp][lane] = make_float4(P.x, P.y, H.x, H.y);
        __syncthreads();
        if (warp == 0) compose(w, comp, cut, fresh, p, col, lane, a.dev_err);
        __syncthreads();
        float2 h = warp_state(comp, cut, warp, lane);
        if (!live) return;
        const int64_t t = t0 + warp * kTok;
        const int left = (int)min((int64_t)kTok, a.T_total - t);
        IO* y = static_cast<IO*>(a.y) + t * a.D + c0;
        float* edge = a.edges + t / kEdge * a.D + c0;
        if ((starts | ends) == 0 && left == kTok) {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                if (k % kEdge == 0 && a.edges) store_pair(edge + (int64_t)(k / kEdge) * a.D, h);
                h = recurrence_next(c[k], nb[k], h);
                if (a.y) store_pair(y, h);
                y += a.D;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                const bool start = starts >> k & 1;
                const int at = warp * kTok + k;
                if (k % kEdge == 0 && a.edges && k < left)
                    store_pair(edge + (int64_t)(k / kEdge) * a.D,
                               !start  ? h
                               : a.h0 ? state_row(a.h0, marks.start_seq[at], a.D, c0)
                                      : both(0.f));
                if (start) h = both(0.f);
                h = recurrence_next(c[k], nb[k], h);
                if (k < left && a.y) store_pair(y, h);
                y += a.D;
                if (k < left && ends >> k & 1 && a.h_out)
                    store_pair(a.h_out + (int64_t)marks.end_seq[at] * a.D + c0, h);
            }
        }
    });
}

// -------------------------------------------------------------- gradients --

template <typename In, typename IO, int kTok, int kStages, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) scan_bwd_kernel(
    const __grid_constant__ RecurrenceArgs a, const __grid_constant__ Shared w,
    const __grid_constant__ GateBound gb) {
    using S = Stage<In, IO, true, kTok>;
    extern __shared__ __align__(128) char ring[];
    __shared__ Compose comp;
    __shared__ Marks<S::kT> marks;
    __shared__ float2 sums[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_dependents_launch();
    if (w.seqs == nullptr) check_sequences(a, blockIdx.x * kC + 2 * lane, a.dh_out, a.dh0);
    for_tiles<S, In, IO, true, kStages>(a, w, ring, [&](const char* st, int p, int row, int col) {
        const int64_t t0 = (int64_t)row * S::kT;
        const int c0 = col * kC + 2 * lane;
        const bool live = c0 < a.D;
        unsigned starts = 0, ends = 0, cut = 0;
        bool fresh = false;
        if (find_marks<S>(a, w, st, row, marks)) {
            starts = marks.starts[warp];
            ends = marks.ends[warp];
            cut = __brev(marks.end_warps) >> (32 - kWarps);  // in the scan's order
            fresh = marks.ends[kWarps - 1] >> (kTok - 1) & 1;
        }
        const ChannelRate r = channel_rate(
            live ? *reinterpret_cast<const float2*>(a.A_log + c0) : both(0.f), gb.g_min);

        // the negated factors of l in the gradients, from the states, and -dy
        float2 c[kTok], fx[kTok], fz[kTok], fi[kTok], dy[kTok];
        float2 h = *reinterpret_cast<const float2*>(st + S::kEdges + (warp * kC + 2 * lane) * 4);
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const int t = warp * kTok + k;
            if (starts >> k & 1)
                h = a.h0 && live ? state_row(a.h0, marks.start_seq[t], a.D, c0) : both(0.f);
            const float2 x = input<S, In>(st, 0, t, lane);
            const StepGrad u = recurrence_grad(x, input<S, In>(st, 1, t, lane),
                                               input<S, In>(st, 2, t, lane), r, gb, h);
            c[k] = u.c;
            fx[k] = u.dx;
            fz[k] = u.dz;
            fi[k] = u.di;
            h = recurrence_next(u.c, mul2(u.dx, x), h);
            dy[k] = mul2(pair(reinterpret_cast<const IO*>(st + S::kDy) + t * kC + 2 * lane), both(-1.f));
            if (k % 2 == 1) asm volatile("" ::: "memory");
        }
        if (ends && a.dh_out) {
            float2 d[kTok];
#pragma unroll
            for (int k = 0; k < kTok; ++k)
                d[k] = ends >> k & 1 && live
                           ? state_row(a.dh_out, marks.end_seq[warp * kTok + k], a.D, c0)
                           : both(0.f);
#pragma unroll
            for (int k = 0; k < kTok; ++k) dy[k] = fma2(d[k], both(-1.f), dy[k]);
        }
        // -r, what -l_t has from later tokens: r_{t-1} = a_t (dy_t + r_t)
        float2 P = both(1.f), H = both(0.f);
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            if (ends >> k & 1) H = both(0.f);
            P = fma2(c[k], P, P);
            const float2 l = add2(dy[k], H);
            H = fma2(c[k], l, l);
        }
        const int turn = kWarps - 1 - warp;  // the warp's place in the scan
        comp.map[turn][lane] = make_float4(P.x, P.y, H.x, H.y);
        __syncthreads();
        if (warp == 0) compose(w, comp, cut, fresh, p, col, lane, a.dev_err);
        __syncthreads();
        float2 nr = warp_state(comp, cut, turn, lane);
        const int64_t t = t0 + warp * kTok;
        const int64_t at = t * a.D + c0;
        const int left = live ? (int)min((int64_t)kTok, a.T_total - t) : 0;
        IO* dx = static_cast<IO*>(a.dx) + at;
        IO* dz = static_cast<IO*>(a.dz) + at;
        IO* di = static_cast<IO*>(a.di) + at;
        float2 dA = both(0.f);
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            if (ends >> k & 1) nr = both(0.f);
            const float2 l = add2(dy[k], nr);
            nr = fma2(c[k], l, l);
            if (k < left) {
                const int64_t o = (int64_t)k * a.D;
                const float2 v = mul2(l, fz[k]);
                store_pair(dx + o, mul2(l, fx[k]));
                store_pair(dz + o, v);
                store_pair(di + o, mul2(l, fi[k]));
                // (an infinite z has a gradient of zero)
                const float2 z = input<S, In>(st, 1, warp * kTok + k, lane);
                dA.x += v.x == 0.f ? 0.f : v.x * z.x;
                dA.y += v.y == 0.f ? 0.f : v.y * z.y;
                if (starts >> k & 1 && a.dh0)
                    store_pair(a.dh0 + (int64_t)marks.start_seq[warp * kTok + k] * a.D + c0,
                               mul2(nr, both(-1.f)));
            }
        }
        if (a.dA_log) {
            sums[warp][lane] = dA;
            __syncthreads();
            if (warp == 0 && live) {
                float2 s = sums[0][lane];
#pragma unroll
                for (int j = 1; j < kWarps; ++j) s = add2(s, sums[j][lane]);
                *reinterpret_cast<float2*>(w.part + (int64_t)row * a.D + c0) = s;
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
        auto next = [&](float2 xe, float2 ze, float2 ie, float2 Ae, float2 he) {
            const Step s = recurrence_step(xe, ze, ie, channel_rate(Ae, 0.f).neg_log2, gb);
            return recurrence_next(s.c, s.nb, he);
        };
        const float2 a = next(make_float2(xv.x, xv.y), make_float2(zv.x, zv.y),
                              make_float2(iv.x, iv.y), make_float2(A.x, A.y), make_float2(v.x, v.y));
        const float2 b = next(make_float2(xv.z, xv.w), make_float2(zv.z, zv.w),
                              make_float2(iv.z, iv.w), make_float2(A.z, A.w), make_float2(v.z, v.w));
        v = make_float4(a.x, a.y, b.x, b.y);
        *hp = v;
    }
    store_four(y + n * D + c, v);
}

// --------------------------------------------------------------- launches --

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// The parts of a workspace for rows of tiles of kT tokens; w may be nullptr.
size_t lay_out(char* ws, int64_t T, int D, int kT, bool bwd, Shared* w, float** edges) {
    const size_t rows = (size_t)((T + kT - 1) / kT), cols = (D + kC - 1) / kC;
    size_t n = 0;
    auto take = [&](size_t bytes) {
        char* p = ws ? ws + n : nullptr;
        n += up(bytes);
        return p;
    };
    Shared s{};
    s.rows = (int)rows;
    s.cols = (int)cols;
    if (bwd) {  // (first, so that a forward before the gradients does not touch them)
        char* e = take((size_t)((T + kEdge - 1) / kEdge) * D * 4);
        if (edges) *edges = reinterpret_cast<float*>(e);
        s.part = reinterpret_cast<float*>(take(rows * D * 4));
    }
    if (rows != 1) {
        s.counter = reinterpret_cast<uint32_t*>(take(8));
        s.seqs = reinterpret_cast<int2*>(take(rows * sizeof(int2)));
        s.mail = reinterpret_cast<ulonglong2*>(take(rows * cols * 64 * sizeof(ulonglong2)));
    }
    if (w) *w = s;
    return n;
}

template <typename S, typename Kernel>
cudaError_t launch_scan(Kernel kernel, const char* name, int smem, int ctas, const RecurrenceArgs& a,
                        const Shared& w, const float* from, float* to) {
    if (w.rows != 1) {
        const int64_t want = std::max<int64_t>((int64_t)w.rows * w.cols * 16, (int64_t)a.N * 32);
        const int grid = (int)std::min<int64_t>((want + 255) / 256, 152 * 8);
        ProfScope prof("recurrence_setup_kernel", a.stream);
        setup_kernel<<<std::max(grid, 1), 256, 0, a.stream>>>(a, w, S::kT, from, to);
    }
    if (w.rows == 0) return cudaGetLastError();
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
        return e;
    // (one row of tiles: a CTA a column, no tickets)
    const int64_t all = (int64_t)w.rows * w.cols;
    const int64_t grid = w.rows == 1 ? all : std::min<int64_t>(all, 152 * ctas);
    ProfScope prof(name, a.stream);
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), smem, a.stream, a, w,
                            gate_bound(a.g_min));
}

// Tokens a warp holds in the forward: what keeps the tile's inputs at 48 KB (and packed inputs' states
// those of the same inputs whole, bit by bit).
template <typename IO>
constexpr int kForwardTok = sizeof(IO) == 4 ? 8 : 16;

template <typename In, typename IO>
cudaError_t forward(const RecurrenceArgs& a, char* ws) {
    constexpr int kTok = kForwardTok<IO>, kStages = sizeof(In) == 1 ? 3 : 2, kCtas = 2;
    using S = Stage<In, IO, false, kTok>;
    Shared w;
    lay_out(ws, a.T_total, a.D, S::kT, false, &w, nullptr);
    return launch_scan<S>(scan_kernel<In, IO, kTok, kStages, kCtas>, "recurrence_kernel",
                          kStages * S::kBytes, kCtas, a, w, a.h0, a.h_out);
}

template <typename In, typename IO>
cudaError_t backward(RecurrenceArgs a) {
    constexpr int kTok = kEdge, kCtas = sizeof(In) == 4 ? 1 : 2, kStages = 3;
    using S = Stage<In, IO, true, kTok>;
    Shared w;
    float* edges;
    char* ws = static_cast<char*>(a.workspace);
    lay_out(ws, a.T_total, a.D, S::kT, true, &w, &edges);
    if (a.edges == nullptr) {
        RecurrenceArgs f = a;
        f.edges = a.edges = edges;
        f.y = nullptr;
        f.h_out = nullptr;
        if (cudaError_t e = forward<In, IO>(f, ws + up((size_t)((a.T_total + kEdge - 1) / kEdge) *
                                                       a.D * 4)))
            return e;
    }
    if (cudaError_t e = launch_scan<S>(scan_bwd_kernel<In, IO, kTok, kStages, kCtas>,
                                       "recurrence_bwd_kernel", kStages * S::kBytes, kCtas, a, w,
                                       a.dh_out, a.dh0))
        return e;
    if (a.dA_log) {
        ProfScope prof("recurrence_rate_kernel", a.stream);
        return launch_dependent(rate_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, a.stream,
                                (const float*)w.part, w.rows, a.D, a.dA_log);
    }
    return cudaGetLastError();
}

}  // namespace

// (of either type: tiles of 64 tokens have the most rows)
size_t recurrence_fwd_workspace_size(int64_t T, int, int D) {
    return lay_out(nullptr, T, D, kEdge * kWarps, false, nullptr, nullptr);
}
size_t recurrence_bwd_workspace_size(int64_t T, int, int D) {
    return lay_out(nullptr, T, D, kEdge * kWarps, true, nullptr, nullptr);
}

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a) {
    char* ws = static_cast<char*>(a.workspace);
    return a.io_bf16 ? forward<__nv_bfloat16, __nv_bfloat16>(a, ws) : forward<float, float>(a, ws);
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
