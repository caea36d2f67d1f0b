// linear_common.cuh -- what the kernels of the per-head-decay linear attention share: the
// problem, the linear-attention call that the forward and all three gradients are instances of,
// and the map from segment slots to token ranges.
//
// One call, with rows x, y of da channels and w of db channels, computes per sequence and head
//     forward:  S_t = e^{g_t} S_{t-1} + y_t w_t^T,                out_t = S_t^T x_t
//     reversed: D_t = e^{g_{t+1}} D_{t+1} + y_t w_t^T,            out_t = D_t^T x_t
//   o  = forward (x, y, w) = (q, k, v)          dq = forward (do, v, k)  (states transposed)
//   dv = reversed (k, q, do)                    dk = reversed (v, do, q) (states transposed)
//
// Segments.  The recurrence is linear, so a sequence is cut into segments of L tokens that run in
// parallel once the state at each segment's edge is known.  Slot base(n) + s holds segment s of
// sequence n, with base(n) = floor(cu[n] / L) + n: consecutive bases are at least ceil(len / L)
// apart, so a slot finds its sequence from cu_seqlens alone and no launch has to lay out a table.
// Slots past a sequence's last segment are empty. Only sequences of more than one segment have
// states at segments' edges.  Where sequences are many these lie more closely: from floor(2 cu[n] /
// L) on, for ceil(len / L) <= floor(2 len / L) where len > L, so that 2 T / L slots hold them
// however many sequences there are.
#pragma once

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace lin {

struct Problem {
    const int32_t* cu;
    int N;
    int64_t T;
    int H;
    const float* g;
    int g_per_token;
    int L;
    int edges;       // slots of edge states
    int edges_close; // nonzero: they begin at floor(2 cu[n] / L), else at the segments' slots
    unsigned* err;
};

struct Call {
    const void *x, *y, *w;
    int64_t x_ld, y_ld, w_ld;
    int da, db;
    int reverse;
    int tr;              // states in memory are [db][da] instead of [da][db]
    const float* edge;   // [N][H][...] state before the first (reversed: after the last) token
    const float* seg;    // [edges][H][...] state at the other segments' edges, or nullptr
    // what follows at a sequence's end (token by token in the outputs' kernel, on the tensor cores
    // in the segment sums' and the edges'):
    float* S_out;        // [N][H][...] state after the sequence (reversed: before it), or nullptr
    const float* anchor; // [N][H][...] states whose dot products with those after the sequences
    float* anchors;      //   are wanted, or nullptr: [N][H][kAnchors] partial sums
    void* out;           // [T][H][db]
    const void* dot;     // [T][H][db] rows, or nullptr: dots[b][h][t] = sum over column block b
    int64_t dot_ld;      //   of out * dot in fp32, before out is rounded and without the token's
    float* dots;         //   own term (x_t . y_t) (w_t . dot_t)
};

constexpr int kMaxCalls = 3, kAnchors = 16;
struct Calls {
    Call c[kMaxCalls];
};

__host__ __device__ inline int64_t slot_count(int64_t T, int N, int L) { return T / L + N; }

// the slot of the edge state of the first segment of sequence n, whose first token is a
__device__ __forceinline__ int edge_base(const Problem& p, uint32_t a, int n) {
    return p.edges_close ? (int)(2 * a / (uint32_t)p.L) : (int)(a / (uint32_t)p.L) + n;
}

struct Segment {
    int n;                // sequence
    int s, count;         // segment of the sequence, and how many it has
    int begin, end;       // its tokens (there are fewer than 2^31)
    int edge;             // (where count > 1) the slot of its edge state
    bool live;
};

__device__ __forceinline__ uint32_t seq_start(const Problem& p, int n) {
    return p.cu ? (uint32_t)__ldg(p.cu + n) : (uint32_t)n * ((uint32_t)p.T / (uint32_t)p.N);
}

// The segment in slot j.  kWarp: called by whole warps, whose lanes search together; else by one
// thread on its own.
template <bool kWarp = true>
__device__ __forceinline__ Segment find_segment(const Problem& p, int j) {
    const int lane = threadIdx.x & 31;
    const uint32_t L = p.L;
    int lo = 0, hi = p.N;  // the sequence is in [lo, hi)
    while (!kWarp && hi - lo > 1) {
        const int n = (lo + hi) / 2;
        if (seq_start(p, n) / L + (uint32_t)n <= (uint32_t)j) lo = n;
        else hi = n;
    }
    while (kWarp && hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int n = lo + (lane + 1) * step;
        const bool at = n < hi && seq_start(p, n) / L + (uint32_t)n <= (uint32_t)j;
        const unsigned mask = __ballot_sync(0xffffffffu, at);
        const int c = mask == 0xffffffffu ? 32 : __ffs(~mask) - 1;
        lo += c * step;
        hi = min(hi, lo + step);
    }
    // (as seq_range(), in 32 bits; a malformed range reads as empty)
    const uint32_t a = seq_start(p, lo);
    const uint32_t b = p.cu ? seq_start(p, lo + 1) : a + (uint32_t)p.T / (uint32_t)p.N;
    const uint32_t T = (uint32_t)p.T;
    const bool bad = p.cu && ((int)a < 0 || b < a || b > T || (lo == 0 && a != 0) ||
                              (lo == p.N - 1 && b != T));
    Segment r;
    r.n = lo;
    r.count = bad ? 0 : (int)((b - a + L - 1) / L);
    r.s = j - (int)((bad ? 0u : a) / L) - lo;
    r.live = r.s >= 0 && r.s < r.count;
    r.begin = (int)(a + (uint32_t)r.s * L);
    r.end = (int)min((uint32_t)r.begin + L, b);
    r.edge = edge_base(p, a, lo) + r.s;
    return r;
}

// The launch's first CTA reports any malformed offset: find_segment() looks at some only.
__device__ __forceinline__ void check_seqlens(const Problem& p) {
    if (p.cu == nullptr) return;
    for (int n = threadIdx.x; n < p.N; n += blockDim.x) {
        int64_t a, b;
        seq_range(p.cu, n, p.N, p.T, p.err, a, b);
    }
}

__device__ __forceinline__ float log_decay(const Problem& p, int64_t t, int h) {
    return p.g_per_token ? __ldg(p.g + t * p.H + h) : __ldg(p.g + h);
}

}  // namespace lin
}  // namespace kda
