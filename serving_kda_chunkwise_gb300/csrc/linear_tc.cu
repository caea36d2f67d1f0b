// linear_tc.cu -- the per-head-decay linear attention of bf16 inputs on the tcgen05 tensor
// cores: the segment sums, the outputs and the final states of a call (linear_common.cuh).
//
// Chunks of C = 128 tokens.  With X, Y [C, da] and W [C, db] the chunk's rows, S the state at
// its start and G the running sum of g inside it (forward; reversed in brackets):
//     A   = (X Y^T) .* D,   D_ri = e^{G_r - G_i} for i <= r   [e^{G_i - G_r} for i >= r]
//     out = A W + Diag(e^{G_r}) X S                           [e^{G_C - G_r}]
//     S  <- e^{G_C} S + Y^T Diag(e^{G_C - G_i}) W             [e^{G_i}]
// (reversed chunks run from the last to the first, S is then the state at the chunk's end).
//
// Precision.  X, Y, W are bf16 as given, so X Y^T is exact up to its fp32 accumulation.  In the
// outputs A, S and the decayed W are held as bf16 hi + lo (16 bits of mantissa, 2^-17) in two
// products each, which is lost in the rounding of the outputs to bf16.  Where fp32 results come of
// them there is a third part, for fp32's 24 bits: of S and the decayed W in the calls whose dot
// products make up the decay's gradient (dg of 65,536 x 16: 2.0e-6 off, with two parts 4.3e-6; a
// third part of A finds no room, and costs heads of short memory 3e-6), and of the decayed W in the
// segment sums, which form all states that are results or that segments start from (2e-7 off; with
// two parts 2.5e-6). No decay is formed as a quotient or as a difference of long sums: with P and U
// a token's prefix and suffix sums inside its block of 32 tokens and B the blocks' sums, every
// exponent is a sum of terms of one sign except inside a diagonal block, where the difference of
// prefix sums is taken on sums kept in two floats.  So nothing overflows, strong decays underflow
// to zero, and a strong token does not cost the weak ones behind it their precision.  A log2 decay
// below -2000 is taken as -2000 (2^-2000 is zero in fp32), which makes g = -inf an exact reset.
#include <cuda.h>

#include "linear_common.cuh"
#include "linear_tc.h"
#include "tc_util.cuh"

namespace kda {
namespace lintc {
namespace {

using namespace tc;
using lin::Call;
using lin::Problem;
using lin::Segment;

constexpr int kC = 128;  // tokens a chunk
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- waits --
// A whole warp waits, and all of its lanes agree on whether it did: after an abort no lane is
// left behind at a later warp-wide step.  The polling loop is kept out of line: each role runs its
// code once a chunk, beside the other roles', and what does not fit the instruction cache costs.
__device__ __noinline__ bool wait_poll(uint64_t* bar, uint32_t parity, unsigned* err,
                                       volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_wait_ab(bar, parity, err, abort));
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, unsigned* err,
                                     volatile int* abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
    return wait_poll(bar, parity, err, abort);
}
// The same by one thread.
__device__ __noinline__ bool wait1(uint64_t* bar, uint32_t parity, unsigned* err,
                                   volatile int* abort) {
    return mbar_wait_ab(bar, parity, err, abort);
}

// hi, lo and what these leave of (a0, a1), in bf16
__device__ __forceinline__ void split3(float a0, float a1, uint32_t& hi, uint32_t& lo,
                                       uint32_t& rest) {
    hi = pack_bf16x2(a0, a1);
    a0 -= __uint_as_float(hi << 16);
    a1 -= __uint_as_float(hi & 0xffff0000u);
    lo = pack_bf16x2(a0, a1);
    rest = pack_bf16x2(a0 - __uint_as_float(lo << 16), a1 - __uint_as_float(lo & 0xffff0000u));
}

// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ void st_shared(float* p, float x) {
    asm volatile("st.shared.f32 [%0], %1;" : : "r"(smem_u32(p)), "f"(x) : "memory");
}
// The registers of earlier TMEM loads are ready (tied to the wait, so that no use moves above it).
__device__ __forceinline__ void landed(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                   "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                   "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void landed(float (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                   "+f"(v[6]), "+f"(v[7])
                 :
                 : "memory");
}
// Warp-collective: 8 consecutive fp32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------- descriptors --
// Operand descriptors (128-byte swizzle, 1024 bytes between 8-row groups) as a constant upper
// word and a lower word that steps by constants.
__device__ __forceinline__ uint32_t dlow(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t low) {
    constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
    return (static_cast<uint64_t>(kHigh) << 32) | low;
}

// ------------------------------------------------- pairs of fp32 numbers --
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}
// bf16 hi of (a0, a1) and of what hi leaves of them
__device__ __forceinline__ void split2(float a0, float a1, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(a0, a1);
    float l0, l1;
    asm("{\n\t.reg .b64 a, h, m;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 h, {%4, %5};\n\t"
        "mov.b64 m, {%6, %6};\n\tfma.rn.f32x2 a, h, m, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(l0), "=f"(l1)
        : "f"(a0), "f"(a1), "f"(__uint_as_float(hi << 16)),
          "f"(__uint_as_float(hi & 0xffff0000u)), "f"(-1.f));
    lo = pack_bf16x2(l0, l1);
}

// ------------------------------------------------------------- work items --
// Items: slots x heads x calls, the calls of one (slot, head) next to each other so that they
// share the rows through L2.
struct Item {
    Segment sg;
    int slot, call, h, chunks;
};

struct OutParams {
    Problem p;
    lin::Calls calls;
    CUtensorMap x[lin::kMaxCalls], y[lin::kMaxCalls], w[lin::kMaxCalls];
    CUtensorMap seg[lin::kMaxCalls], edge[lin::kMaxCalls];  // states (outputs only)
    int n_calls;
    int slots;
    const float* rec;  // decay records, see decay_kernel
    unsigned* next;    // how many items have been taken beyond the first round
    int sums;          // which (kSegments, kSingles)
};

__device__ __forceinline__ uint32_t item_count(const OutParams& o) {
    return (uint32_t)o.slots * o.p.H * o.n_calls;
}

// By one thread; out of line, once an item.
__device__ __noinline__ Item item_at(const OutParams& o, uint32_t i) {
    Item t;
    t.call = (int)(i % o.n_calls);
    i /= o.n_calls;
    t.h = (int)(i % o.p.H);
    t.slot = (int)(i / o.p.H);
    t.sg = lin::find_segment<false>(o.p, t.slot);
    t.chunks = t.sg.live ? (t.sg.end - t.sg.begin + kC - 1) / kC : 0;
    return t;
}

// The c-th chunk of the walk: its place in the segment, first token and length.
struct Chunk {
    int i, t0, len;
};

// ---------------------------------------------------------------- decays --
// What a chunk's decays are needed as, formed once for all calls and roles: a record of floats a
// (chunk, head), arrays of 128 tokens.  The records lie by slots of one chunk.
constexpr int kRP = 0, kRPlo = 128;   // prefix sum inside the block of 32 (log2), its rounding
constexpr int kRU = 256;              // exclusive suffix sum inside the block
constexpr int kRHead = 384;           // 2^(sum from the chunk's start, inclusive)
constexpr int kRTail = 512;           // 2^(sum to the chunk's end, exclusive)
// forward, then reversed: column factors for the blocks beside the diagonal (2^U, 2^P) and for
// the diagonal's (2^-P, 2^P), the four blocks' sums, their total
constexpr int kRCol = 640, kRB = 256, kRDir = 264;
constexpr int kRec = 1184;

// One warp a (chunk, head); a CTA's warps take neighbouring heads, whose decays share sectors.
// Bound by writing the records (4.7 KB each): 27 us at 65,536 tokens x 32 heads, 2.9 TB/s.  (The
// output kernel's own warps formed them before, and each chunk waited for them.)
__global__ void __launch_bounds__(256) decay_kernel(const __grid_constant__ Problem p, float* rec,
                                                    unsigned* next) {
    grid_dependents_launch();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kCounters) next[threadIdx.x] = 0u;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * 8 + (threadIdx.x >> 5);
    // blocks are slots of one chunk, for most of a segment's chunks may lie past a short sequence
    Problem chunks = p;
    chunks.L = kC;
    const Segment sg = lin::find_segment(chunks, (int)blockIdx.x);
    if (h >= p.H || !sg.live) return;
    const int t0 = sg.begin;
    float* r = rec + ((size_t)blockIdx.x * p.H + h) * kRec;
    float e[4], P[4], Plo[4], U[4], B[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int t = t0 + 32 * b + lane;
        const float x = t < sg.end ? lin::log_decay(p, t, h) * kLog2e : 0.f;
        e[b] = x < -2000.f ? -2000.f : x;  // (a NaN stays one)
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        float x = e[b], lo = 0.f;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, x, off);
            const float ylo = __shfl_up_sync(0xffffffffu, lo, off);
            if (lane >= off) {  // (x, lo) += (y, ylo), the rounding of x + y kept in lo
                const float s = __fadd_rn(x, y), d = __fsub_rn(s, x);
                const float err = __fadd_rn(__fsub_rn(x, __fsub_rn(s, d)), __fsub_rn(y, d));
                x = s;
                lo = __fadd_rn(__fadd_rn(lo, ylo), err);
            }
        }
        P[b] = x;
        Plo[b] = lo;
        B[b] = __shfl_sync(0xffffffffu, x, 31);
        float u = __shfl_down_sync(0xffffffffu, e[b], 1);
        if (lane == 31) u = 0.f;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, u, off);
            if (lane + off < 32) u += y;
        }
        U[b] = u;
    }
    const float before[4] = {0.f, B[0], B[0] + B[1], B[0] + B[1] + B[2]};
    const float after[4] = {B[1] + B[2] + B[3], B[2] + B[3], B[3], 0.f};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int i = 32 * b + lane;
        r[kRP + i] = P[b];
        r[kRPlo + i] = Plo[b];
        r[kRU + i] = U[b];
        r[kRHead + i] = ex2f(P[b] + before[b]);
        r[kRTail + i] = ex2f(U[b] + after[b]);
        r[kRCol + i] = ex2f(U[b]);
        // (2^-lo and 2^lo: a factor of the diagonal block is up to 2^24 and its product with a
        // row's about 1, so that the rounding of P would be seen)
        const float lo = 0.6931471805599453f * Plo[b];
        r[kRCol + 128 + i] = ex2f(-P[b]) * (1.f - lo);
        r[kRCol + kRDir + i] = r[kRCol + kRDir + 128 + i] = ex2f(P[b]) * (1.f + lo);
    }
    if (lane < 2) {
        float* s = r + kRCol + lane * kRDir + kRB;
        *reinterpret_cast<float4*>(s) = make_float4(B[0], B[1], B[2], B[3]);
        s[4] = (B[0] + B[1]) + (B[2] + B[3]);
    }
}

// -------------------------------------------------------------- outputs --
// Persistent, one CTA an SM.  Roles: warps 0..7 turn X Y^T into A (hi + lo over the product's own
// TMEM columns, so that A never leaves tensor memory) and write half of the outputs; warps 8..15
// keep the state's copy, write the other half and decay W; a thread each of warps 16..18 loads X
// and the decays (and finds the items), Y, and W and the items' states (as lanes of one warp they
// held each other up by up to 2500 cycles); one of warp 19 issues the MMAs.  Warp w reaches TMEM
// lanes 32 (w % 4) .. + 31.  The state lives in TMEM in fp32; X S reads its bf16 hi + lo copy in
// shared memory.
// Shared memory holds one chunk of X, Y and W (32 KB each), the decayed W and the state's copy (64
// KB each): no second stage fits, but each operand is reloaded as soon as its last product is
// done, and while one waits the others' products run.  (Two stages fit with 64 of the db columns
// to a CTA; that form made A twice and its N = 64 products run at 75 % of N = 128's rate, and was
// slower.)
// Bound by that chain: a chunk takes 8,900 cycles, of which the products are 4,400.  Measured at
// 65,536 tokens x 32 heads x 128: 547 us (2.2 GB at 4.0 TB/s, 7 products of 4.2 MFLOP a chunk
// and head at 880 TFLOP/s); gradients, 65,536 x 16: 1,130 us, dq and dk with dot products and third
// parts (9 products) and dv without.  Items are taken as CTAs come to them (packed prompts of 17 to
// 5,753 tokens x 16: 215 us; dealt out they took a fifth longer).
constexpr int kThreads = 640;
constexpr int kMmaT = 19 * 32;
constexpr uint32_t kSX = 0, kSY = 32768, kSW = 65536;
constexpr uint32_t kSWd = 98304;             // decayed W: hi, lo
constexpr uint32_t kSS = kSWd + 65536;       // state: hi, lo
constexpr uint32_t kSRec = kSS + 65536;      // the record's part for the call's direction
constexpr uint32_t kSOwn = kSRec + 1088;     // the diagonal of X Y^T, of two chunks
constexpr uint32_t kSItem = kSOwn + 1024;    // this item's facts and the next one's
constexpr uint32_t kSBar = kSItem + 128;
constexpr uint32_t kOutSmem = kSBar + 256;
static_assert(kOutSmem <= 232448, "shared-memory limit");
// TMEM columns (all 512 are allocated, so the base address is 0): X Y^T / A, A W, X S, state
constexpr uint32_t kTA = 0, kTO1 = 128, kTO2 = 256, kTS = 384;

struct OutBars {
    uint64_t x, y, w, rec;   // operands and decays loaded
    uint64_t sc, a;          // X Y^T complete; A written (8 arrivals)
    uint64_t s, wd;          // state and its copy written; decayed W written (8 arrivals each)
    uint64_t upd, xs, aw;    // state update, X S, A W complete
    uint64_t read;           // the chunk's outputs (dots: and W) read (16 arrivals)
    uint64_t stored;         // ... and read from their stage (16 arrivals)
    uint64_t item[2];        // an item's facts are there
    uint64_t used[2];        // ... and done with (19 arrivals)
    uint64_t idle;           // the last item's state is done with (8 arrivals)
    uint64_t open, taken;    // the item's state loaded; all of it taken over (8 arrivals)
    uint64_t own[2];         // (dots) the chunk's diagonal of X Y^T written (4 arrivals)
    uint64_t drain;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(OutBars) <= 256, "barrier area");

// What the warps need of an item, kept in shared memory: their registers are few, and what the
// compiler would put into local memory comes back from L2 (shared memory takes all of L1).  One
// thread finds it, an item ahead: by each warp for itself an item began 4000 cycles later.  Items
// are taken as CTAs come to them, for their lengths differ.
struct View {
    volatile int* v;
    enum { kBegin, kEnd, kChunks, kCall, kH, kRev, kRecord, kZero, kN, kSeg, kState, kWords };
    __device__ __forceinline__ int chunks() const { return v[kChunks]; }
    __device__ __forceinline__ int call() const { return v[kCall]; }
    __device__ __forceinline__ int h() const { return v[kH]; }
    __device__ __forceinline__ int rev() const { return v[kRev]; }
    __device__ __forceinline__ Chunk chunk(int k) const {
        Chunk c;
        c.i = v[kRev] ? v[kChunks] - 1 - k : k;
        c.t0 = v[kBegin] + c.i * kC;
        c.len = min(v[kEnd] - c.t0, kC);
        return c;
    }
    __device__ __forceinline__ const float* record(const OutParams& o, int k) const {
        const int i = v[kRev] ? v[kChunks] - 1 - k : k;
        return o.rec + ((size_t)(v[kRecord] + i) * o.p.H + v[kH]) * kRec;
    }
};
__device__ __forceinline__ View view(uint8_t* sm, uint32_t n) {
    return View{reinterpret_cast<volatile int*>(sm + kSItem) + 12 * (n & 1)};
}
static_assert(2 * 12 * 4 <= kSBar - kSItem && View::kWords <= 12, "items' facts");
__device__ __forceinline__ void put_item(const OutParams& o, const Item& t, View w) {
    const int rev = o.calls.c[t.call].reverse;
    w.v[View::kBegin] = t.sg.begin;
    w.v[View::kEnd] = t.sg.end;
    w.v[View::kChunks] = t.chunks;
    w.v[View::kCall] = t.call;
    w.v[View::kH] = t.h;
    w.v[View::kRev] = rev;
    w.v[View::kRecord] = (t.sg.begin - t.sg.s * o.p.L) / kC + t.sg.n + t.sg.s * (o.p.L / kC);
    w.v[View::kZero] = t.sg.count <= 1 && o.calls.c[t.call].edge == nullptr;
    w.v[View::kN] = t.sg.n;
    // the state that it starts from: a segment's edge state or the sequence's own
    w.v[View::kSeg] = t.sg.count > 1;
    w.v[View::kState] = (t.sg.count > 1 ? t.sg.edge : t.sg.n) * o.p.H + t.h;
}

// One operand's loads (0: X and the decays, 1: Y, 2: W), by one thread: chunk after chunk, each
// once the last chunk's buffer has been read.  Returns the number of chunks loaded.
template <bool kDots>
__device__ __noinline__ int load_operand(const OutParams& o, OutBars& bar, int which, uint8_t* sm) {
    const CUtensorMap* maps = which == 0 ? o.x : which == 1 ? o.y : o.w;
    uint8_t* dst = sm + (which == 0 ? kSX : which == 1 ? kSY : kSW);
    uint64_t* full = which == 0 ? &bar.x : which == 1 ? &bar.y : &bar.w;
    uint64_t* freed = which == 0 ? &bar.xs : which == 1 ? &bar.upd : &bar.aw;
    volatile int* abort = &bar.abort;
    unsigned* err = o.p.err;
    const uint32_t items = item_count(o);
    int g = 0;
    uint32_t states = 0, i = blockIdx.x;
    for (uint32_t n = 0;; ++n) {
        const View it = view(sm, n);
        if (which == 0) {
            if (n > 0) {
                if (n == 1) grid_dependency_wait();
                i = gridDim.x + atomicAdd(o.next, 1u);
            }
            if (n > 1 && !wait1(&bar.used[n & 1], ((n >> 1) - 1) & 1, err, abort)) return g;
            if (i < items) put_item(o, item_at(o, i), it);
            else it.v[View::kChunks] = -1;
            mbar_arrive(&bar.item[n & 1]);
        } else if (!wait1(&bar.item[n & 1], (n >> 1) & 1, err, abort)) {
            return g;
        }
        const int chunks = it.chunks(), call = it.call(), h = it.h();
        if (chunks < 0) return g;
        const Call& c = o.calls.c[call];
        const int blocks = (which == 2 ? c.db : c.da) / 64;
        for (int k = 0; k < chunks; ++k, ++g) {
            const uint32_t last = (g - 1) & 1;
            if (which == 2 && k == 0) {  // the item's state, through its copy's buffer
                const CUtensorMap* m = (it.v[View::kSeg] ? o.seg : o.edge) + call;
                const int inner = c.tr ? c.da : c.db, bytes = (c.tr ? c.db : c.da) * 128;
                const int at = it.v[View::kState], boxes = it.v[View::kZero] ? 0 : inner / 32;
                if (states == 0) grid_dependency_wait();
                if (states > 0) {
                    // into L2 early: all CTAs come to their next items at about the same time
#pragma unroll 1
                    for (int b = 0; b < boxes; ++b) tma_prefetch_3d(m, 32 * b, 0, at);
                    if (!wait1(&bar.idle, (states - 1) & 1, err, abort)) return g;
                }
                if (boxes) mbar_expect_tx(&bar.open, boxes * bytes);
                else mbar_arrive(&bar.open);
#pragma unroll 1
                for (int b = 0; b < boxes; ++b)
                    tma_load_3d(sm + kSS + b * bytes, m, 32 * b, 0, at, &bar.open);
                // (it has landed before this thread can come to any way out)
                mbar_wait(&bar.open, states & 1, nullptr);
                ++states;
            }
            if (g > 0 && !wait1(freed, last, err, abort)) return g;
            // (dots: the outputs take their own terms from W)
            if (which == 2 && g > 0 && !wait1(kDots ? &bar.read : &bar.wd, last, err, abort))
                return g;
            const Chunk ch = it.chunk(k);
            mbar_expect_tx(full, blocks * 16384);
#pragma unroll 1
            for (int b = 0; b < blocks; ++b)
                tma_load_3d(dst + b * 16384, maps + call, 64 * b, h, ch.t0, full);
            if (which == 2 && k + 1 < chunks) {  // its load is waited for longest: into L2 early
                const int ahead = it.chunk(k + 1).t0;
#pragma unroll 1
                for (int b = 0; b < blocks; ++b)
                    tma_prefetch_3d(maps + call, 64 * b, h, ahead);
            }
            if (which == 0) {
                if (g > 0 && !wait1(&bar.a, last, err, abort)) return g + 1;
                if (g == 0) grid_dependency_wait();
                mbar_expect_tx(&bar.rec, 4 * kRDir);
                bulk_g2s(sm + kSRec, it.record(o, k) + kRCol + (c.reverse ? kRDir : 0), 4 * kRDir,
                         &bar.rec);
            }
        }
        if (which != 0) mbar_arrive(&bar.used[n & 1]);
    }
}

// The item's state from the buffer that the copy is to have, where 32-float boxes of its rows in
// memory lie (128 bytes a row, 16-byte pieces permuted by the row), into TMEM.
__device__ __noinline__ void load_state(const OutParams& o, uint8_t* sm, uint32_t n) {
    const View it = view(sm, n);
    const Call& c = o.calls.c[it.call()];
    const uint8_t* buf = sm + kSS;
    const int col = threadIdx.x >= 384 ? 64 : 0;
    const int lane = threadIdx.x & 31, row = threadIdx.x & 127;
    const uint32_t to = (static_cast<uint32_t>(row & 96) << 16) + kTS + col;
    const bool zero = it.v[View::kZero] || col >= c.db || (row & 96) >= c.da;
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
        uint32_t u[16];
        if (zero) {
#pragma unroll
            for (int x = 0; x < 16; ++x) u[x] = 0u;
        } else if (c.tr) {
            const uint8_t* f = buf + (row >> 5) * c.db * 128 + (col + 16 * b) * 128 + (lane & 3) * 4;
#pragma unroll
            for (int x = 0; x < 16; ++x)
                u[x] = *reinterpret_cast<const uint32_t*>(f + x * 128 + ((lane >> 2 ^ (x & 7)) << 4));
        } else {
            const uint8_t* f = buf + ((col >> 5) + (b >> 1)) * c.da * 128 + row * 128;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                reinterpret_cast<uint4*>(u)[x] = *reinterpret_cast<const uint4*>(
                    f + ((4 * (b & 1) + x ^ (row & 7)) << 4));
        }
        tmem_st16(to + 16 * b, u);
    }
    tmem_st_wait();
    __syncwarp();
}

// Outputs of one chunk, 32 columns from `col` of one row a lane: rowf (X S) + A W, and for kDots
// their dot products with another row.  A is then without its diagonal, and the token's own term,
// x . y w, joins the outputs after the dot product.  A warp's 32 rows are its TMEM lanes: stored
// from there, each access would touch 32 lines and keep the load/store unit busy for 2000 cycles,
// so a warp passes its 2 KB through the decayed W's buffer (whose product is complete, and which
// the next chunk's overwrites only then).  A TMA store of the whole tile kept that buffer for
// 2200 cycles.
template <bool kDots>
__device__ __forceinline__ bool write_out(const OutParams& o, OutBars& bar, uint8_t* sm,
                                          uint32_t g, View it, int k, float rowf, int col) {
    const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
    const Call& c = o.calls.c[it.call()];
    const int db = c.db, h = it.h();
    const Chunk ch = it.chunk(k);
    const bool cols = col < db, dots = kDots && cols && row < ch.len;
    // (the other rows' first pieces early, while the products are waited for)
    const uint4* dr = nullptr;
    uint4 d[2];
    if (dots) {
        dr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.dot) +
                                            (int64_t)(ch.t0 + row) * c.dot_ld + h * db + col);
        d[0] = __ldg(dr);
        d[1] = __ldg(dr + 1);
    }
    const uint32_t phase = g & 1;
    if (!wait(&bar.aw, phase, o.p.err, &bar.abort) ||
        !wait(&bar.xs, phase, o.p.err, &bar.abort) ||
        !wait(&bar.upd, phase, o.p.err, &bar.abort) ||
        (kDots && !wait(&bar.own[phase], (g >> 1) & 1, o.p.err, &bar.abort)))
        return false;
    tc_fence_after();
    const float own =
        kDots ? reinterpret_cast<const float*>(sm + kSOwn)[128 * phase + row] : 0.f;
    const uint32_t from = (static_cast<uint32_t>(row & 96) << 16) + col;
    uint8_t* stage = sm + kSWd + (col >> 6) * 16384;
    const int piece = (col & 32) >> 3;  // of 16 bytes, within the 128 of a row
    float acc = 0.f;
    // 16 columns at a time, to stay within the registers.  With dots one after the other: unrolled
    // they spilled (1,083 against 1,026 us at 65,536 x 16).  Without them unrolled (561 against 584
    // us at 65,536 x 32).
#pragma unroll (kDots ? 1 : 2)
    for (int b = 0; b < 2; ++b) {
        float o1[16];
        if (cols) {
            float o2[8];
            tmem_ld16(from + kTO1 + 16 * b, o1);
            tmem_ld8(from + kTO2 + 16 * b, o2);
            landed(o1);
            landed(o2);
#pragma unroll
            for (int x = 0; x < 8; ++x) o1[x] = fmaf(rowf, o2[x], o1[x]);
            tmem_ld8(from + kTO2 + 16 * b + 8, o2);
            landed(o2);
#pragma unroll
            for (int x = 0; x < 8; ++x) o1[8 + x] = fmaf(rowf, o2[x], o1[8 + x]);
        }
        if (!kDots && b == 1) {  // the accumulators may be written again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.read);
        }
        if (dots) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t u[4] = {d[x].x, d[x].y, d[x].z, d[x].w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    acc = fmaf(o1[8 * x + 2 * y], __uint_as_float(u[y] << 16), acc);
                    acc = fmaf(o1[8 * x + 2 * y + 1], __uint_as_float(u[y] & 0xffff0000u), acc);
                }
                if (b == 0) d[x] = __ldg(dr + 2 + x);
                // the row of W, which stays in its buffer until `read`
                const uint4 w = *reinterpret_cast<const uint4*>(
                    sm + kSW + (col >> 6) * 16384 + row * 128 +
                    ((piece + 2 * b + x) ^ (row & 7)) * 16);
                const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    float &a0 = o1[8 * x + 2 * y], &a1 = o1[8 * x + 2 * y + 1];
                    a0 = fmaf(own, __uint_as_float(v[y] << 16), a0);
                    a1 = fmaf(own, __uint_as_float(v[y] & 0xffff0000u), a1);
                }
            }
        }
        if (kDots && b == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.read);
        }
        if (!cols) continue;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float* v = o1 + 8 * x;
            *reinterpret_cast<uint4*>(stage + row * 128 + ((piece + 2 * b + x) ^ (row & 7)) * 16) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
    }
    if (dots) c.dots[((int64_t)(col >> 5) * o.p.H + h) * o.p.T + ch.t0 + row] = acc;
    __syncwarp();
    // four lanes a row; rows 4 apart share a phase, for their pieces lie in different banks
    const int r0 = (row & 96) + (lane >> 3) + (lane & 4);
    uint4 u[4];
    if (cols)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + 8 * j;
            u[j] = *reinterpret_cast<const uint4*>(stage + r * 128 +
                                                   ((piece + (lane & 3)) ^ (r & 7)) * 16);
        }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.stored);
    if (cols) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(c.out) +
                             ((int64_t)(ch.t0 + r0) * o.p.H + h) * db + col + 8 * (lane & 3);
        const int64_t step = (int64_t)8 * o.p.H * db;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r0 + 8 * j < ch.len) *reinterpret_cast<uint4*>(out + j * step) = u[j];
    }
    return true;
}

// kDots: the calls want their outputs' dot products, and have third parts of the state's copy and
// of the decayed W.  Those have no buffers of their own: the copy's lies in the decayed W's lo
// part's until X S is done, W's then in the copy's.  (Calls without them are launched on their own:
// in one kernel for both, 1,319 us against 1,130 for the gradients of 65,536 x 16.)
template <bool kDots>
__global__ void __launch_bounds__(kThreads, 1) out_kernel(const __grid_constant__ OutParams o) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    OutBars& bar = *reinterpret_cast<OutBars*>(sm + kSBar);
    const Problem& p = o.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bar.abort;
    if (tid == 0) {
        uint64_t* one[] = {&bar.x,  &bar.y,   &bar.w,  &bar.rec, &bar.sc,
                           &bar.upd, &bar.xs, &bar.aw, &bar.drain};
        for (uint64_t* b : one) mbar_init(b, 1);
        mbar_init(&bar.open, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bar.item[b], 1);
            mbar_init(&bar.used[b], 19);
            mbar_init(&bar.own[b], 4);
        }
        uint64_t* eight[] = {&bar.a, &bar.s, &bar.wd, &bar.idle, &bar.taken};
        for (uint64_t* b : eight) mbar_init(b, 8);
        mbar_init(&bar.read, 16);
        mbar_init(&bar.stored, 16);
        fence_mbar_init();
        bar.abort = 0;
    }
    if (warp == 0) tmem_alloc(&bar.tmem, 512);
    if (blockIdx.x == 0) lin::check_seqlens(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int loads = 0;  // chunks loaded by this thread (for the way out of an abort)
    grid_dependents_launch();
    if (warp < 16) grid_dependency_wait();  // (X, Y and W are no earlier launch's)

    if (warp >= 16 && warp < 19) {
        if (lane == 0) loads = load_operand<kDots>(o, bar, warp - 16, sm);
    } else if (tid == kMmaT) {
        // ------------------------------------------------------- MMA thread
        constexpr uint32_t id_sc = idesc_bf16(128, 128, false, false);  // X Y^T
        const uint32_t lX = dlow(sbase + kSX, 0), lYk = dlow(sbase + kSY, 0);
        const uint32_t lYm = dlow(sbase + kSY, 16384), lW = dlow(sbase + kSW, 16384);
        const uint32_t lWd = dlow(sbase + kSWd, 16384), lS = dlow(sbase + kSS, 16384);
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t i = 0;; ++i) {
            if (!wait1(&bar.item[i & 1], (i >> 1) & 1, p.err, abort)) break;
            const View it = view(sm, i);
            const int chunks = it.chunks(), call = it.call();
            if (chunks < 0) break;
            const int da = o.calls.c[call].da;
            const uint32_t n = (uint32_t)(o.calls.c[call].db >> 3) << 17;   // N = db
            const uint32_t id_out = (idesc_bf16(128, 0, false, true)) | n;  // A W, X S
            const uint32_t id_up = (idesc_bf16(128, 0, true, true)) | n;    // Y^T W
            for (int k = 0; ok && k < chunks; ++k, ++g) {
                const uint32_t ph = g & 1;
                ok = wait1(&bar.x, ph, p.err, abort) && wait1(&bar.y, ph, p.err, abort);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    if (ks == 4 && da == 64) break;
                    const uint32_t off = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                    mma_bf16(kTA, desc(lX + off), desc(lYk + off), id_sc, ks > 0);
                }
                mma_commit(&bar.sc);
                // X S and the state's update as soon as their operands are there, then A W: the
                // longest way round is from the update through the next Y and X Y^T to A (A W
                // first: 9.8k cycles a chunk).  With the decayed W the rows past a chunk that
                // ends inside its tile are cleared, too.
                uint32_t todo = 7;
                uint64_t since = 0;
                while (todo) {
                    uint32_t now = 0;
                    const bool free = g == 0 || test(&bar.read, ph ^ 1);
                    if ((todo & 3) && test(&bar.s, ph)) {
                        if ((todo & 1) && test(&bar.wd, ph)) now = 1;
                        else if ((todo & 2) && free) now = 2;
                    }
                    if (now == 0 && (todo & 5) == 4 && free && test(&bar.a, ph))
                        now = 4;
                    if (now == 0) {
                        if (since == 0) since = globaltimer();
                        if (*abort) { ok = false; break; }
                        if (globaltimer() - since > kWaitLimitNs) {
                            atomicOr(p.err, kDevErrTimeout);
                            *abort = 1;
                            ok = false;
                            break;
                        }
                        continue;
                    }
                    todo &= ~now;
                    since = 0;
                    tc_fence_after();
                    if (now == 1) {
                        // S += Y^T Wd: 128 tokens in 8 steps, hi and lo (da = 64: the second 64
                        // lanes take whatever the buffer's second half holds, never read)
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                mma_bf16(kTS, desc(lYm + (ks * 2048 >> 4)),
                                         desc(lWd + ((part * 32768 + ks * 2048) >> 4)), id_up, 1);
                        if (kDots)  // (the third part from the state's copy's buffer)
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)
                                mma_bf16(kTS, desc(lYm + (ks * 2048 >> 4)),
                                         desc(lS + (ks * 2048 >> 4)), id_up, 1);
                        mma_commit(&bar.upd);
                    } else if (now == 2) {
                        // X S
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            if (ks == 4 && da == 64) break;
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                mma_bf16(kTO2,
                                         desc(lX + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4)),
                                         desc(lS + ((part * 32768 + ks * 2048) >> 4)), id_out,
                                         ks + part > 0);
                        }
                        if (kDots)  // (from the decayed W's lo part's buffer)
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks) {
                                if (ks == 4 && da == 64) break;
                                mma_bf16(kTO2,
                                         desc(lX + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4)),
                                         desc(lWd + ((32768 + ks * 2048) >> 4)), id_out, 1);
                            }
                        mma_commit(&bar.xs);
                    } else {
                        // A W: A's 16-token steps are 8 columns of hi and 8 of lo
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                mma_bf16_ts(kTO1, kTA + 16 * ks + 8 * part,
                                            desc(lW + (ks * 2048 >> 4)), id_out, ks + part > 0);
                        mma_commit(&bar.aw);
                    }
                }
            }
            if (!ok) break;
            mbar_arrive(&bar.used[i & 1]);
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ A warps
        const int q = warp & 3, wg = warp >> 2;
        const uint32_t at = static_cast<uint32_t>(32 * q) << 16 | kTA;
        const float* rCol = reinterpret_cast<const float*>(sm + kSRec);
        const int row = 32 * q + lane;
        uint32_t g = 0, n = 0;
        bool ok = true;
        for (; ok; ++n) {
            if (!wait(&bar.item[n & 1], (n >> 1) & 1, p.err, abort)) break;
            const View it = view(sm, n);
            if (it.chunks() < 0) break;
            // the row's factor in the diagonal block, which is a column's of the other direction,
            // and its sum to the edge of the block that it looks to, loaded a chunk ahead (from
            // memory they take 2500 cycles)
            float diag_next = 0.f, edge_next = 0.f;
            if (it.chunks()) {
                const float* r = it.record(o, 0);
                diag_next = __ldg(r + kRCol + (it.rev() ? 0 : kRDir) + 128 + row);
                edge_next = __ldg(r + (it.rev() ? kRU : kRP) + row);
            }
#pragma unroll 1
            for (int k = 0; k < it.chunks(); ++k, ++g) {
                const int rev = it.rev();
                const int len = it.chunk(k).len;
                const float diag = diag_next, edge = edge_next;
                if (k + 1 < it.chunks()) {
                    const float* r = it.record(o, k + 1);
                    diag_next = __ldg(r + kRCol + (rev ? 0 : kRDir) + 128 + row);
                    edge_next = __ldg(r + (rev ? kRU : kRP) + row);
                }
                if (!wait(&bar.rec, g & 1, p.err, abort) || !wait(&bar.sc, g & 1, p.err, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // blocks at distance n from the diagonal: 0 and 3, or 1 and 2 (no warp has more
                // than two inside the triangle)
#pragma unroll 1
                for (int m = 0; m < 2; ++m) {
                    const int n = wg == 0 ? 3 * m : 1 + m;
                    const int j = rev ? q + n : q - n, z = rev ? q - n : q + n;
                    if (n > 0 && z >= 0 && z < 4) {  // outside the triangle
                        uint32_t zero[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) zero[c] = 0u;
                        tmem_st32(at + 32 * z, zero);
                    }
                    if (j < 0 || j > 3) continue;
                    // Columns that count: all of a block beside the diagonal but those past the
                    // segment, on the diagonal those of the triangle.
                    uint32_t in = 0xffffffffu;
                    if (rev && len - 32 * j < 32)
                        in = len > 32 * j ? (1u << (len - 32 * j)) - 1u : 0u;
                    if (n == 0) in &= rev ? ~((1u << lane) - 1u) : (2u << lane) - 1u;
                    if (n == 0 && kDots) in &= ~(1u << lane);
                    // The row's decay up to the block times the columns' inside it.  On the
                    // diagonal these are 2^P_r and 2^-P_i (reversed: 2^-P_r, 2^P_i), at most 2^24,
                    // formed from sums kept in two floats.
                    const bool strong = n == 0 && !(rCol[kRB + q] > -24.f);
                    float x = edge;
                    if (n > 1) x += rCol[kRB + (rev ? q + 1 : q - 1)];
                    if (n > 2) x += rCol[kRB + (rev ? q + 2 : q - 2)];
                    const float rf = n == 0 ? diag : ex2f(x);
                    const float* cf = rCol + (n == 0 ? 128 : 0) + 32 * j;
#pragma unroll 1
                    for (int hf = 0; hf < 2; ++hf) {  // 16 columns, a step of A W
                        float v[16];
                        tmem_ld16(at + 32 * j + 16 * hf, v);
                        landed(v);
                        if (kDots && n == 0) {
                            // (a store each: picked by index, the values went to local memory)
                            float* own = reinterpret_cast<float*>(sm + kSOwn) + 128 * (g & 1) + row;
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (lane == 16 * hf + c) st_shared(own, v[c]);
                        }
                        if (!strong) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                float4 f = reinterpret_cast<const float4*>(cf + 16 * hf)[c];
                                mul2(f.x, f.y, rf, rf);
                                mul2(f.z, f.w, rf, rf);
                                mul2(v[4 * c], v[4 * c + 1], f.x, f.y);
                                mul2(v[4 * c + 2], v[4 * c + 3], f.z, f.w);
                            }
                        } else {
                            // strong decays: the difference of the prefix sums, kept in two floats
                            const float sgn = rev ? -1.f : 1.f;
                            const float p_hi = __ldg(it.record(o, k) + kRP + row);
                            const float p_lo = __ldg(it.record(o, k) + kRPlo + row);
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const float hi = __shfl_sync(0xffffffffu, p_hi, 16 * hf + c);
                                const float lo = __shfl_sync(0xffffffffu, p_lo, 16 * hf + c);
                                v[c] *= ex2f(sgn * ((p_hi - hi) + (p_lo - lo)));
                            }
                        }
                        if (n == 0 || in != 0xffffffffu) {
                            const uint32_t part = in >> (16 * hf);
#pragma unroll
                            for (int c = 0; c < 16; ++c) v[c] = part & (1u << c) ? v[c] : 0.f;
                        }
                        uint32_t u[16];  // 8 columns of hi, 8 of lo
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            split2(v[2 * c], v[2 * c + 1], u[c], u[c + 8]);
                        tmem_st16(at + 32 * j + 16 * hf, u);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kDots && wg == 0) mbar_arrive(&bar.own[g & 1]);
                    mbar_arrive(&bar.a);
                }
                // the second half of its 64 output columns (the state warps write the first)
                const float rowf = __ldg(it.record(o, k) + (it.rev() ? kRTail : kRHead) + row);
                ok = write_out<kDots>(o, bar, sm, g, it, k, rowf, 64 * wg + 32);
                if (!ok) break;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.used[n & 1]);
        }
    } else if (warp < 16) {
        // --------------------------------------- state, decayed W and outputs
        const int q = warp & 3, wg = (warp - 8) >> 2;
        const int row = 32 * q + lane;  // token, or state row
        const uint32_t at = (static_cast<uint32_t>(32 * q) << 16) + 64 * wg;  // this warp's columns
        uint32_t g = 0, opened = 0, n = 0;
        bool ok = true;
        for (; ok; ++n) {
            if (!wait(&bar.item[n & 1], (n >> 1) & 1, p.err, abort)) break;
            const View it = view(sm, n);
            if (it.chunks() < 0) break;
            if (it.chunks() == 0) {
                if (lane == 0) mbar_arrive(&bar.used[n & 1]);
                continue;
            }
            const bool cols = 64 * wg < o.calls.c[it.call()].db;          // this warp has columns
            const bool holds = cols && row < o.calls.c[it.call()].da;     // this lane a state row
            float rowf_prev = 0.f, head, tail, total;
            {
                const float* r = it.record(o, 0);
                head = __ldg(r + kRHead + row);
                tail = __ldg(r + kRTail + row);
                total = __ldg(r + kRCol + kRB + 4);
            }
            if (!wait(&bar.open, opened & 1, p.err, abort)) { ok = false; break; }
            tc_fence_after();
            load_state(o, sm, n);
            // no warp writes the copy while another still reads the buffer
            if (lane == 0) mbar_arrive(&bar.taken);
            if (!wait(&bar.taken, opened & 1, p.err, abort)) { ok = false; break; }
            ++opened;
            // step k: the outputs of chunk k - 1 and the state's copy of chunk k, then chunk k's
            // decayed W (the outputs' products were the last to read W's buffer, so its load runs
            // meanwhile)
#pragma unroll 1
            for (int k = 0; k <= it.chunks(); ++k) {
                const int rev = it.rev();
                const float rowf = rev ? tail : head, wf = rev ? head : tail, all = ex2f(total);
                if (k + 1 < it.chunks()) {  // the next chunk's, early
                    const float* r = it.record(o, k + 1);
                    head = __ldg(r + kRHead + row);
                    tail = __ldg(r + kRTail + row);
                    total = __ldg(r + kRCol + kRB + 4);
                }
                if (k < it.chunks()) {
                    // the last update of the state, the last read of its copy and of the decayed
                    // W's buffer are complete
                    if (g > 0 && (!wait(&bar.upd, (g - 1) & 1, p.err, abort) ||
                                  !wait(&bar.xs, (g - 1) & 1, p.err, abort))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (cols) {
                        uint8_t* sr = sm + kSS + wg * 16384 + row * 128;
                        // (few columns at a time, to stay within the registers)
                        constexpr int kN = kDots ? 8 : 16;
#pragma unroll 1
                        for (int b = 0; b < 64 / kN; ++b) {
                            float S[kN];
                            if constexpr (kDots) tmem_ld8(at + kTS + kN * b, S);
                            else tmem_ld16(at + kTS + kN * b, S);
                            landed(S);
                            if (holds)
#pragma unroll
                                for (int x = 0; x < kN / 8; ++x) {
                                    const float* v = S + 8 * x;
                                    const uint32_t to = ((kN / 8 * b + x) ^ (row & 7)) << 4;
                                    uint32_t hi[4], lo[4], rest[4];
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        if (kDots) split3(v[2 * y], v[2 * y + 1], hi[y], lo[y], rest[y]);
                                        else split2(v[2 * y], v[2 * y + 1], hi[y], lo[y]);
                                    *reinterpret_cast<uint4*>(sr + to) =
                                        make_uint4(hi[0], hi[1], hi[2], hi[3]);
                                    *reinterpret_cast<uint4*>(sr + 32768 + to) =
                                        make_uint4(lo[0], lo[1], lo[2], lo[3]);
                                    if (kDots)  // (in the decayed W's lo part's buffer)
                                        *reinterpret_cast<uint4*>(sr + (kSWd + 32768 - kSS) + to) =
                                            make_uint4(rest[0], rest[1], rest[2], rest[3]);
                                }
                            uint32_t u[kN];
#pragma unroll
                            for (int x = 0; x < kN; x += 2) {
                                mul2(S[x], S[x + 1], all, all);
                                u[x] = __float_as_uint(S[x]);
                                u[x + 1] = __float_as_uint(S[x + 1]);
                            }
                            if constexpr (kDots) tmem_st8(at + kTS + kN * b, u);
                            else tmem_st16(at + kTS + kN * b, u);
                        }
                        tmem_st_wait();
                        fence_async_smem();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.s);
                }
                if (k == it.chunks()) {
                    // the last reads of the copy's buffer are complete: the next item's state may
                    // come
                    if (!wait(&bar.xs, (g - 1) & 1, p.err, abort) ||
                        (kDots && !wait(&bar.upd, (g - 1) & 1, p.err, abort))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive(&bar.idle);
                }
                if (k > 0 && !write_out<kDots>(o, bar, sm, g - 1, it, k - 1, rowf_prev, 64 * wg)) {
                    ok = false;
                    break;
                }
                if (k < it.chunks()) {
                    if (!wait(&bar.w, g & 1, p.err, abort) ||
                        (g > 0 && !wait(&bar.stored, (g - 1) & 1, p.err, abort)) ||
                        (kDots && !wait(&bar.xs, g & 1, p.err, abort))) {
                        ok = false;
                        break;
                    }
                    const int len = it.chunk(k).len;
                    const bool dead = row >= len;
                    if (cols) {
                        const uint8_t* wr = sm + kSW + wg * 16384 + row * 128;
                        uint8_t* wd = sm + kSWd + wg * 16384 + row * 128;
                        constexpr int kN = kDots ? 2 : 4;
#pragma unroll 1
                        for (int b = 0; b < 8 / kN; ++b) {
                            uint4 in[kN];
#pragma unroll
                            for (int x = 0; x < kN; ++x)
                                in[x] = *reinterpret_cast<const uint4*>(
                                    wr + (((kN * b + x) ^ (row & 7)) << 4));
                            if (dead)
#pragma unroll
                                for (int x = 0; x < kN; ++x) in[x] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int x = 0; x < kN; ++x) {
                                const uint32_t w[4] = {in[x].x, in[x].y, in[x].z, in[x].w};
                                uint32_t hi[4], lo[4], rest[4];
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    float a0 = __uint_as_float(w[y] << 16);
                                    float a1 = __uint_as_float(w[y] & 0xffff0000u);
                                    mul2(a0, a1, wf, wf);
                                    if (kDots) split3(a0, a1, hi[y], lo[y], rest[y]);
                                    else split2(a0, a1, hi[y], lo[y]);
                                }
                                const uint32_t to = ((kN * b + x) ^ (row & 7)) << 4;
                                *reinterpret_cast<uint4*>(wd + to) =
                                    make_uint4(hi[0], hi[1], hi[2], hi[3]);
                                *reinterpret_cast<uint4*>(wd + 32768 + to) =
                                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
                                if (kDots)  // (in the state's copy's buffer, which has been read)
                                    *reinterpret_cast<uint4*>(wd + (kSS - kSWd) + to) =
                                        make_uint4(rest[0], rest[1], rest[2], rest[3]);
                            }
                        }
                    }
                    if (len < kC) {
                        // rows past the segment hold another sequence's tokens (or zeros): they
                        // must not reach a product even as 0 * inf.  (X Y^T is masked instead.)
                        if (!wait(&bar.y, g & 1, p.err, abort)) { ok = false; break; }
                        if (dead) {
                            uint4* wr = reinterpret_cast<uint4*>(sm + kSW + wg * 16384 + row * 128);
                            uint4* yr = reinterpret_cast<uint4*>(sm + kSY + wg * 16384 + row * 128);
#pragma unroll 1
                            for (int x = 0; x < 8; ++x)  // (each lane from another piece: other banks)
                                wr[(x + lane) & 7] = yr[(x + lane) & 7] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.wd);
                    ++g;
                }
                rowf_prev = rowf;
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.used[n & 1]);
        }
    }

    __syncthreads();
    if (bar.abort) {
        // let copies and MMAs still in flight land before leaving
        if (loads > 0) {
            mbar_wait(warp == 16 ? &bar.x : warp == 17 ? &bar.y : &bar.w, (loads - 1) & 1, nullptr);
            // (where the abort came before the last chunk's decays were asked for, this wait runs
            // out, by when those of the chunk before have landed)
            if (warp == 16) mbar_wait(&bar.rec, (loads - 1) & 1, nullptr);
        }
        if (tid == kMmaT) {
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, nullptr);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

// --------------------------------------------------------- segment sums --
// sum_i e^{G_end - G_i} y_i w_i^T over a segment [reversed: e^{G_i} from its start]: for the scan
// over a sequence's segments, or of a sequence that is one segment (or empty), which with the state
// before it is the state after it.  W is decayed in place (hi over W itself, lo and the third part
// beside it); two stages of all operands fit but for the third part, which waits until the last
// chunk's products are done with its buffer. A tensor core adds to its accumulator by truncation,
// 4e-8 of it a step: the small parts have an accumulator of their own, the chunks take turns at
// three for hi, and the walk is towards the edge that the weights refer to, so that what counts
// most comes last.  (Away from it, into one accumulator for all parts, with two parts of W: <S, D>
// of heads that remember a thousand tokens was 1e-5 off.) Bound by reading Y and W, and by the
// conversion of W between a stage's load and its products: 241 us at 65,536 tokens x 32 heads x
// 128, 1.07 GB at 4.5 TB/s (with two parts of W 209 us, without the conversion 176); packed prompts
// with states 108 us; 256 x 300 tokens x 32 heads with states, where an item is three chunks and a
// state in and out, 541 us, 2.3 GB at 4.3 TB/s.
constexpr int kSumThreads = 640;
constexpr uint32_t kUY = 0, kUW = 32768, kULo = 65536, kUStage = 98304;  // two stages
constexpr uint32_t kUThird = 2 * kUStage;
constexpr uint32_t kUItem = kUThird + 32768;
constexpr uint32_t kUBar = kUItem + 128;
constexpr uint32_t kSumSmem = kUBar + 256;
static_assert(kSumSmem <= 232448, "shared-memory limit");
// TMEM columns (all 512): three accumulators of hi, one of lo and the third part
constexpr uint32_t kUSmall = 384;
constexpr int kUTurns = 3;

struct SumBars {
    uint64_t full[2], done[2], wd[2], drain;
    uint64_t item[2], used[2];  // as in OutBars (17 arrivals)
    uint32_t tmem;
    int abort;
};

__global__ void __launch_bounds__(kSumThreads, 1) sum_kernel(const __grid_constant__ OutParams o,
                                                             float* dec) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    SumBars& bar = *reinterpret_cast<SumBars*>(sm + kUBar);
    const Problem& p = o.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bar.abort;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.done[i], 1);
            mbar_init(&bar.wd[i], 16);
            mbar_init(&bar.item[i], 1);
            mbar_init(&bar.used[i], 17);
        }
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
        bar.abort = 0;
    }
    if (warp == 0) tmem_alloc(&bar.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependents_launch();
    const uint32_t items = item_count(o);
    // an item whose sum nothing needs, or none in this launch (a walk's last segment is needed only
    // for the state after the sequence; an empty sequence owns its first slot)
    auto skip = [&](const Item& t) {
        const Call& c = o.calls.c[t.call];
        const bool final = c.S_out || c.anchor;
        if (t.sg.count <= 1)
            return !(o.sums & kSingles) || !final || (t.sg.count == 0 ? t.sg.s != 0 : !t.sg.live);
        const bool last = c.reverse ? t.sg.s == 0 : t.sg.s == t.sg.count - 1;
        return !(o.sums & kSegments) || !t.sg.live || (last && !final);
    };
    int loads = 0;  // stages loaded by the TMA thread (for the way out of an abort)

    auto view = [&](uint32_t n) {
        return View{reinterpret_cast<volatile int*>(sm + kUItem) + 12 * (n & 1)};
    };

    if (warp == 0) {
        // Items are taken some at a time, as CTAs come to them: where most sequences are shorter
        // than a segment most items have no sum, and a lane each finds that out.
        const uint32_t some = min(32u, 1 + items / (8 * gridDim.x));
        uint32_t g = 0, n = 0;
        bool ok = true;
        for (uint32_t round = 0; ok; ++round) {
            uint32_t base = blockIdx.x;
            if (round > 0) {
                if (round == 1) grid_dependency_wait();
                if (lane == 0) base = gridDim.x + atomicAdd(o.next, 1u);
                base = __shfl_sync(0xffffffffu, base, 0);
            }
            base *= some;
            if (base >= items) break;
            Item t{};
            bool has = lane < some && base + lane < items;
            if (has) {
                t = item_at(o, base + lane);
                has = !skip(t);
            }
            for (uint32_t mask = __ballot_sync(0xffffffffu, has); ok && mask; mask &= mask - 1) {
                if (n > 1 && !wait(&bar.used[n & 1], ((n >> 1) - 1) & 1, p.err, abort)) {
                    ok = false;
                    break;
                }
                const View it = view(n);
                if (lane == __ffs(mask) - 1) put_item(o, t, it);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.item[n & 1]);
                    const int call = it.call(), h = it.h();
                    const Call& c = o.calls.c[call];
                    if (c.edge && !it.v[View::kSeg]) {  // read at the item's end: into L2 early
                        const int64_t E = (int64_t)c.da * c.db;
                        l2_prefetch(c.edge + ((int64_t)it.v[View::kN] * p.H + h) * E, 4 * E);
                    }
                    for (int k = 0; k < it.chunks(); ++k, ++g) {
                        const uint32_t st = g & 1;
                        if (g >= 2 && !wait1(&bar.done[st], ((g - 2) >> 1) & 1, p.err, abort)) {
                            ok = false;
                            break;
                        }
                        const Chunk ch = it.chunk(k);
                        uint8_t* s = sm + st * kUStage;
                        mbar_expect_tx(&bar.full[st], (c.da + c.db) / 64 * 16384);
#pragma unroll 1
                        for (int b = 0; b < c.da / 64; ++b)
                            tma_load_3d(s + kUY + b * 16384, &o.y[call], 64 * b, h, ch.t0,
                                        &bar.full[st]);
#pragma unroll 1
                        for (int b = 0; b < c.db / 64; ++b)
                            tma_load_3d(s + kUW + b * 16384, &o.w[call], 64 * b, h, ch.t0,
                                        &bar.full[st]);
                        loads = (int)g + 1;
                        if (k + 2 < it.chunks()) {  // its stage comes free late: into L2 early
                            const int ahead = it.chunk(k + 2).t0;
#pragma unroll 1
                            for (int b = 0; b < c.da / 64; ++b)
                                tma_prefetch_3d(&o.y[call], 64 * b, h, ahead);
#pragma unroll 1
                            for (int b = 0; b < c.db / 64; ++b)
                                tma_prefetch_3d(&o.w[call], 64 * b, h, ahead);
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                ++n;
            }
        }
        if (ok && (n < 2 || wait(&bar.used[n & 1], ((n >> 1) - 1) & 1, p.err, abort)) &&
            lane == 0) {
            view(n).v[View::kChunks] = -1;
            mbar_arrive(&bar.item[n & 1]);
        }
    } else if (tid == 32) {
        const uint32_t lY = dlow(sbase + kUY, 16384), lHi = dlow(sbase + kUW, 16384);
        const uint32_t lLo = dlow(sbase + kULo, 16384), lThird = dlow(sbase + kUThird, 16384);
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            if (!wait1(&bar.item[n & 1], (n >> 1) & 1, p.err, abort)) break;
            const View it = view(n);
            const int chunks = it.chunks();
            if (chunks < 0) break;
            const uint32_t id =
                idesc_bf16(128, 0, true, true) | (uint32_t)(o.calls.c[it.call()].db >> 3) << 17;
            mbar_arrive(&bar.used[n & 1]);
            for (int k = 0; k < chunks; ++k, ++g) {
                const uint32_t st = g & 1;
                if (!wait1(&bar.wd[st], (g >> 1) & 1, p.err, abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t at = st * kUStage >> 4, turn = 128 * (k % kUTurns);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t step = ks * 2048 >> 4;
                    mma_bf16(turn, desc(lY + at + step), desc(lHi + at + step), id,
                             k >= kUTurns || ks > 0);
                    mma_bf16(kUSmall, desc(lY + at + step), desc(lLo + at + step), id, k + ks > 0);
                    mma_bf16(kUSmall, desc(lY + at + step), desc(lThird + step), id, 1);
                }
                mma_commit(&bar.done[st]);
            }
        }
    } else if (warp >= 4) {
        grid_dependency_wait();  // (Y and W are no earlier launch's)
        // 16 warps decay W, each 32 tokens of 32 columns (8 warps took longer than the loads)
        const int q = warp & 3, cg = (warp - 4) >> 2;
        const int row = 32 * q + lane;
        const uint32_t lb = static_cast<uint32_t>(32 * q) << 16;
        uint32_t g = 0;
        // An item's first loads from the decays' records, before the item before it is stored: the
        // chunks' summed log2 decays, chunk k's in lane k (a segment has at most 16), and the row's
        // factor in the first chunk.
        float total = 0.f, first = 0.f;
        auto open = [&](uint32_t n) {
            if (!wait(&bar.item[n & 1], (n >> 1) & 1, p.err, abort)) return false;
            const View it = view(n);
            const int chunks = it.chunks();
            const int mine = (it.rev() ? kRHead : kRTail) + row;
            total = lane < chunks ? __ldg(it.record(o, lane) + kRCol + kRB + 4) : 0.f;
            first = chunks > 0 ? __ldg(it.record(o, 0) + mine) : 0.f;
            return true;
        };
        bool ok = open(0);
        for (uint32_t n = 0; ok; ++n) {
            const View it = view(n);
            const int chunks = it.chunks();
            if (chunks < 0) break;
            const Call& c = o.calls.c[it.call()];
            const int rev = c.reverse;
            const bool cols = 32 * cg < c.db;
            const int mine = (rev ? kRHead : kRTail) + row;
            // log2 decays between the edge and the walk's chunks, and over all of them
            float between = total, next = first;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float x = __shfl_down_sync(0xffffffffu, between, off);
                if (lane + off < 32) between += x;
            }
            const float whole = __shfl_sync(0xffffffffu, between, 0);
            between = __shfl_down_sync(0xffffffffu, between, 1);  // (lane 31's is none's)
#pragma unroll 1
            for (int k = 0; k < chunks; ++k, ++g) {
                const uint32_t st = g & 1;
                const float wf = next * ex2f(__shfl_sync(0xffffffffu, between, k));
                if (k + 1 < chunks) next = __ldg(it.record(o, k + 1) + mine);  // early
                if (!wait(&bar.full[st], (g >> 1) & 1, p.err, abort)) { ok = false; break; }
                uint8_t* stage = sm + st * kUStage;
                const bool dead = row >= it.chunk(k).len;
                const uint32_t own = (cg >> 1) * 16384 + row * 128;
                auto at = [&](int x) { return own + (((4 * (cg & 1) + x) ^ (row & 7)) << 4); };
                uint4 rest[4];
                if (cols) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        rest[x] = *reinterpret_cast<const uint4*>(stage + kUW + at(x));
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t w[4] = {rest[x].x, rest[x].y, rest[x].z, rest[x].w};
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            if (dead) w[y] = 0u;
                            float a0 = __uint_as_float(w[y] << 16);
                            float a1 = __uint_as_float(w[y] & 0xffff0000u);
                            mul2(a0, a1, wf, wf);
                            split3(a0, a1, hi[y], lo[y], w[y]);
                        }
                        *reinterpret_cast<uint4*>(stage + kUW + at(x)) =
                            make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(stage + kULo + at(x)) =
                            make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        rest[x] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (dead) {
                    uint4* yr = reinterpret_cast<uint4*>(stage + kUY + (cg >> 1) * 16384 + row * 128);
#pragma unroll 1
                    for (int x = 0; x < 4; ++x)
                        yr[(4 * (cg & 1) + x) ^ (row & 7)] = make_uint4(0u, 0u, 0u, 0u);
                }
                // the last chunk's products have read their third part
                if (g > 0 && !wait(&bar.done[st ^ 1], ((g - 1) >> 1) & 1, p.err, abort)) {
                    ok = false;
                    break;
                }
                if (cols)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        *reinterpret_cast<uint4*>(sm + kUThird + at(x)) = rest[x];
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.wd[st]);
            }
            if (!ok || !(ok = open(n + 1))) break;
            // The warp's piece of the state: 32 rows x 32 columns, a row a lane in TMEM, four rows
            // an access in memory (where rows lie 4 db bytes apart).  It passes through what the
            // warp itself writes of both stages' lo buffers, 64 bytes of its rows in each.
            const bool piece = cols && 32 * q < c.da, single = !it.v[View::kSeg];
            const int64_t E = (int64_t)c.da * c.db;
            const int64_t at0 = (int64_t)(32 * q + (lane >> 3)) * c.db + 32 * cg + 4 * (lane & 7);
            const int64_t seq = ((int64_t)it.v[View::kN] * p.H + it.h()) * E + at0;
            float4 before[8];  // the state before the segment (S_out may be in its place)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                before[x] = piece && single && c.edge
                                ? *reinterpret_cast<const float4*>(c.edge + seq + 4 * x * c.db)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            // the accumulators are complete with the item's last chunk; the next item's first MMA
            // follows this warp's next arrival
            const uint32_t gl = g - 1;
            if (chunks > 0 && !wait(&bar.done[gl & 1], (gl >> 1) & 1, p.err, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float dot = 0.f;
            auto stage_at = [&](int r, int c16) {
                return reinterpret_cast<float4*>(sm + (c16 >> 2) * kUStage + kULo +
                                                 (cg >> 1) * 16384 + (32 * q + r) * 128 +
                                                 (((4 * (cg & 1) + (c16 & 3)) ^ (r & 7)) << 4));
            };
            if (piece) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float v[8], w[kUTurns][8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] = w[0][x] = w[1][x] = w[2][x] = 0.f;
                    const uint32_t from = lb + 32 * cg + 8 * b;
                    if (chunks > 0) tmem_ld8(from + kUSmall, v);
#pragma unroll
                    for (int turn = 0; turn < kUTurns; ++turn)
                        if (chunks > turn) tmem_ld8(from + 128 * turn, w[turn]);
                    landed(v);
#pragma unroll
                    for (int turn = 0; turn < kUTurns; ++turn) landed(w[turn]);
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] += w[0][x] + (w[1][x] + w[2][x]);
                    *stage_at(lane, 2 * b) = make_float4(v[0], v[1], v[2], v[3]);
                    *stage_at(lane, 2 * b + 1) = make_float4(v[4], v[5], v[6], v[7]);
                }
                __syncwarp();
                auto sum = [&](int x) { return *stage_at(4 * x + (lane >> 3), lane & 7); };
                if (!single) {
                    float* to = const_cast<float*>(c.seg) + it.v[View::kState] * E + at0;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *reinterpret_cast<float4*>(to + 4 * x * c.db) = sum(x);
                } else {
                    const float f = ex2f(whole);
#pragma unroll
                    for (int x = 4; x < 8; ++x)
                        before[x] = c.edge ? *reinterpret_cast<const float4*>(c.edge + seq +
                                                                              4 * x * c.db)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        float4 v = sum(x);
                        v.x = fmaf(f, before[x].x, v.x);
                        v.y = fmaf(f, before[x].y, v.y);
                        v.z = fmaf(f, before[x].z, v.z);
                        v.w = fmaf(f, before[x].w, v.w);
                        if (c.S_out) *reinterpret_cast<float4*>(c.S_out + seq + 4 * x * c.db) = v;
                        if (c.anchor) {
                            const float4 u =
                                __ldg(reinterpret_cast<const float4*>(c.anchor + seq + 4 * x * c.db));
                            dot = fmaf(v.x, u.x, fmaf(v.y, u.y, fmaf(v.z, u.z, fmaf(v.w, u.w, dot))));
                        }
                    }
                }
            }
            if (c.anchor && single) {
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
                if (lane == 0)
                    c.anchors[((int64_t)it.v[View::kN] * p.H + it.h()) * lin::kAnchors + warp - 4] = dot;
            }
            if (!single && warp == 4 && lane == 0)
                dec[(int64_t)rev * p.edges * p.H + it.v[View::kState]] = whole;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.used[n & 1]);
        }
    }

    __syncthreads();
    if (bar.abort) {
        if (tid == 0)
            for (int x = max(loads - 2, 0); x < loads; ++x)
                mbar_wait(&bar.full[x & 1], (x >> 1) & 1, nullptr);
        if (tid == 32) {
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, nullptr);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

// ------------------------------------------------------------------- host --

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// [T][H][d] with a token stride of ld elements: boxes of 64 channels x 1 head x 128 tokens
bool make_map(CUtensorMap* m, const void* base, int64_t T, int H, int d, int64_t ld) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, kC};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 states [count][rows][inner]: boxes of 32 columns x all rows (64 or 128) of one
bool make_state_map(CUtensorMap* m, const void* base, int64_t count, int rows, int inner) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)count};
    const cuuint64_t strides[2] = {(cuuint64_t)inner * 4, (cuuint64_t)rows * inner * 4};
    const cuuint32_t box[3] = {32, (cuuint32_t)rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 1;
}

cudaError_t fill(OutParams& o, const Problem& p, const lin::Calls& calls, int n, int64_t slots,
                 const float* rec, bool out) {
    o.p = p;
    o.calls = calls;
    o.n_calls = n;
    o.slots = (int)slots;
    o.rec = rec;
    for (int i = 0; i < n; ++i) {
        const Call& c = calls.c[i];
        if (p.T == 0) continue;
        if ((out && !make_map(&o.x[i], c.x, p.T, p.H, c.da, c.x_ld)) ||
            !make_map(&o.y[i], c.y, p.T, p.H, c.da, c.y_ld) ||
            !make_map(&o.w[i], c.w, p.T, p.H, c.db, c.w_ld))
            return cudaErrorInvalidValue;
        const int rows = c.tr ? c.db : c.da, inner = c.tr ? c.da : c.db;
        if (out && ((c.seg && !make_state_map(&o.seg[i], c.seg, (int64_t)p.edges * p.H, rows, inner)) ||
                    (c.edge && !make_state_map(&o.edge[i], c.edge, (int64_t)p.N * p.H, rows,
                                               inner))))
            return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

}  // namespace

size_t record_bytes(int64_t T, int N, int H) {
    return (size_t)lin::slot_count(T, N, kC) * H * kRec * sizeof(float);
}

cudaError_t launch_decays(const Problem& p, float* rec, unsigned* next, cudaStream_t s) {
    ProfScope prof("linear_decay_kernel", s);
    const dim3 grid((unsigned)lin::slot_count(p.T, p.N, kC), (p.H + 7) / 8);
    decay_kernel<<<grid, 256, 0, s>>>(p, rec, next);
    return cudaGetLastError();
}

cudaError_t launch_outputs(const Problem& p, const lin::Calls& calls, int n, int64_t slots,
                           const float* rec, unsigned* next, const char* name, cudaStream_t s) {
    OutParams o{};
    o.next = next;
    if (cudaError_t e = fill(o, p, calls, n, slots, rec, true)) return e;
    const auto kernel = calls.c[0].dot ? out_kernel<true> : out_kernel<false>;
    if (cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kOutSmem))
        return e;
    const int64_t items = slots * p.H * n, sms = sm_count();
    ProfScope prof(name, s);
    return launch_dependent(kernel, dim3((unsigned)(items < sms ? items : sms)), dim3(kThreads),
                            kOutSmem, s, o);
}

cudaError_t launch_sums(const Problem& p, const lin::Calls& calls, int n, int64_t slots,
                        const float* rec, float* dec, unsigned* next, int sums,
                        const char* name, cudaStream_t s) {
    OutParams o{};
    o.next = next;
    o.sums = sums;
    if (cudaError_t e = fill(o, p, calls, n, slots, rec, false)) return e;
    if (cudaError_t e = cudaFuncSetAttribute(
            sum_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSumSmem))
        return e;
    const int64_t items = slots * p.H * n, sms = sm_count();
    ProfScope prof(name, s);
    return launch_dependent(sum_kernel, dim3((unsigned)(items < sms ? items : sms)),
                            dim3(kSumThreads), kSumSmem, s, o, dec);
}

}  // namespace lintc
}  // namespace kda
