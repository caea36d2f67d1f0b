// linear_tc.cu -- the per-head-decay linear attention of bf16 inputs on the tcgen05 tensor
// cores: the segment sums and the outputs of a call (linear_common.cuh).
//
// Chunks of C = 128 tokens.  With X, Y [C, da] and W [C, db] the chunk's rows, S the state at
// its start and G the running sum of g inside it (forward; reversed in brackets):
//     A   = (X Y^T) .* D,   D_ri = e^{G_r - G_i} for i <= r   [e^{G_i - G_r} for i >= r]
//     out = A W + Diag(e^{G_r}) X S                           [e^{G_C - G_r}]
//     S  <- e^{G_C} S + Y^T Diag(e^{G_C - G_i}) W             [e^{G_i}]
// (reversed chunks run from the last to the first, S is then the state at the chunk's end).
//
// Precision.  X, Y, W are bf16 as given, so X Y^T is exact up to its fp32 accumulation.  A, S
// and the decayed W are held as bf16 hi + lo (16 bits of mantissa, 2^-17) in two products each:
// with hi alone the fp32 state and the decay's gradient would carry bf16's 2^-9.
// No decay is formed as a quotient or as a difference of long sums: with P and U a token's
// prefix and suffix sums inside its block of 32 tokens and B the blocks' sums, every exponent is
// a sum of terms of one sign except inside a diagonal block, where the difference of prefix sums
// is taken on sums kept in two floats.  So nothing overflows, strong decays underflow to zero,
// and a strong token does not cost the weak ones behind it their precision.  A log2 decay below
// -2000 is taken as -2000 (2^-2000 is zero in fp32), which makes g = -inf an exact reset.
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

// The registers of earlier TMEM loads are ready (tied to the wait, so that no use moves above it).
__device__ __forceinline__ void landed(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                   "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                   "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void landed(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                   "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                   "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                   "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                   "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
                 :
                 : "memory");
    asm volatile("" : "+f"(v[30]), "+f"(v[31]) : : "memory");
}

// ---------------------------------------------------------------- MMAs --
// Issued by the one lane with `lead` set out of warp-uniform code: loop control and descriptors
// then stay in uniform registers (from a branch on the lane every operand of every MMA is moved
// there first, which held the issue to one MMA in 150 cycles).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(lead)
        : "memory");
}
// The same value in every lane, known as such to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// ---------------------------------------------------------------- decays --
// Log decays of the chunk's tokens 32 b + lane, b = 0..3, as they are in memory (loaded a chunk
// ahead); tokens past the segment do not decay.
__device__ __forceinline__ void load_decays(const Problem& p, int t0, int len, int h, int lane,
                                            float (&e)[4]) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int i = 32 * b + lane;
        e[b] = i < len ? lin::log_decay(p, t0 + i, h) : 0.f;
    }
}

__device__ __forceinline__ float pick(const float (&x)[4], int q) {
    return q == 0 ? x[0] : q == 1 ? x[1] : q == 2 ? x[2] : x[3];
}

struct Sums {
    float B[4];  // block sums
    float P, U;  // of this lane's token of block q: inclusive prefix, exclusive suffix
    float Plo;   // P's rounding error (filled by sums<true>)
};

template <bool kTwo>
__device__ __forceinline__ Sums sums(const float (&g)[4], int q, int lane) {
    Sums r;
    float e[4];  // log2 decays
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float x = g[b] * kLog2e;
        e[b] = x < -2000.f ? -2000.f : x;
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        float x = e[b];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        r.B[b] = x;
    }
    const float own = pick(e, q);
    float x = own, lo = 0.f;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, x, off);
        if (kTwo) {  // (x, lo) += (y, ylo), the rounding of x + y kept in lo
            const float ylo = __shfl_up_sync(0xffffffffu, lo, off);
            if (lane >= off) {
                const float s = __fadd_rn(x, y), d = __fsub_rn(s, x);
                const float err = __fadd_rn(__fsub_rn(x, __fsub_rn(s, d)), __fsub_rn(y, d));
                x = s;
                lo = __fadd_rn(__fadd_rn(lo, ylo), err);
            }
        } else if (lane >= off) {
            x += y;
        }
    }
    r.P = x;
    r.Plo = lo;
    float u = __shfl_down_sync(0xffffffffu, own, 1);
    if (lane == 31) u = 0.f;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, u, off);
        if (lane + off < 32) u += y;
    }
    r.U = u;
    return r;
}

// Sum of the blocks before (after) block q, nearest first.
__device__ __forceinline__ float before(const Sums& s, int q) {
    float x = 0.f;
#pragma unroll
    for (int b = 2; b >= 0; --b) x += b < q ? s.B[b] : 0.f;
    return x;
}
__device__ __forceinline__ float after(const Sums& s, int q) {
    float x = 0.f;
#pragma unroll
    for (int b = 1; b < 4; ++b) x += b > q ? s.B[b] : 0.f;
    return x;
}

// ------------------------------------------------------------- work items --
// Items: slots x heads x calls x halves of the call's db columns (64 each), the halves and the
// calls of one (slot, head) next to each other so that they share the rows through L2.
struct Item {
    Segment sg;
    int slot;
    int call, h, half, chunks;
    bool live;
};

struct OutParams {
    Problem p;
    lin::Calls calls;
    CUtensorMap x[lin::kMaxCalls], y[lin::kMaxCalls], w[lin::kMaxCalls];
    int n_calls, halves;
    int64_t slots;
    int wide_store;  // every output row piece is 32-byte aligned
};

__device__ __forceinline__ int64_t item_count(const OutParams& o) {
    return o.slots * o.p.H * o.n_calls * o.halves;
}

__device__ __forceinline__ Item item_at(const OutParams& o, int64_t i) {
    Item t;
    t.half = (int)(i % o.halves);
    i /= o.halves;
    t.call = (int)(i % o.n_calls);
    i /= o.n_calls;
    t.h = (int)(i % o.p.H);
    t.slot = (int)(i / o.p.H);
    t.sg = lin::find_segment(o.p, t.slot);
    t.live = t.sg.live && t.half * 64 < o.calls.c[t.call].db;
    t.chunks = t.live ? (int)((t.sg.end - t.sg.begin + kC - 1) / kC) : 0;
    return t;
}

// First token and length of the c-th chunk of the walk.
__device__ __forceinline__ void chunk_at(const Item& t, int reverse, int c, int& t0, int& len) {
    const int i = reverse ? t.chunks - 1 - c : c;
    t0 = t.sg.begin + i * kC;
    len = min(t.sg.end - t0, kC);
}

// -------------------------------------------------------------- outputs --
// Persistent, one CTA an SM.  Roles: warps 0..3 turn X Y^T into A (hi + lo over the product's own
// TMEM columns, so that A never leaves tensor memory), warp 12 issues the TMA loads (two stages),
// warp 13 the MMAs, and warps 4..11 decay W, convert the state and write the outputs.  Warp w
// reaches TMEM lanes 32 (w % 4) .. + 31.  The state lives in TMEM in fp32; X S reads its bf16
// hi + lo copy in shared memory.
// A CTA takes 64 of the db columns: two full stages of X, Y and W then fit beside the decayed W
// and the state, at the price of forming A twice for db = 128.
constexpr int kThreads = 448;
constexpr uint32_t kSX = 0, kSY = 32768, kSW = 65536, kStage = 81920;  // two stages
constexpr uint32_t kSWd = 2 * kStage;       // decayed W: hi, lo (16 KB each)
constexpr uint32_t kSS = kSWd + 32768;      // state: hi, lo (16 KB each)
constexpr uint32_t kSCol = kSS + 32768;     // column factors, two chunks of 128 floats
constexpr uint32_t kSDiag = kSCol + 1024;   // diagonals of X Y^T, three chunks of 128 floats
constexpr uint32_t kSBar = kSDiag + 1536;
constexpr uint32_t kOutSmem = kSBar + 256;
static_assert(kOutSmem <= 232448, "shared-memory limit");
// TMEM columns: X Y^T / A two buffers of 128, A W 64, X S two of 64, state 64
constexpr uint32_t kTA = 0, kTO1 = 256, kTO2 = 320, kTS = 448;

struct OutBars {
    uint64_t full[2], done[2];   // stage loaded; every MMA of the stage's chunk complete
    uint64_t sc[2], a[2];        // X Y^T complete; A written (4 arrivals)
    uint64_t col[2];             // column factors written (4 arrivals)
    uint64_t s, wd;              // state and its copy written; decayed W written (8 arrivals each)
    uint64_t upd, qs;            // state update complete; X S complete
    uint64_t o_full, o_free;     // chunk's outputs complete; read (8 arrivals)
    uint64_t drain;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(OutBars) <= 256, "barrier area");

__global__ void __launch_bounds__(kThreads, 1) out_kernel(const __grid_constant__ OutParams o) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    OutBars& bar = *reinterpret_cast<OutBars*>(sm + kSBar);
    const Problem& p = o.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bar.abort;
    static_assert(kC == 128, "a chunk is the 128 lanes of a TMEM tile");
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.done[i], 1);
            mbar_init(&bar.sc[i], 1);
            mbar_init(&bar.a[i], 4);
            mbar_init(&bar.col[i], 4);
        }
        mbar_init(&bar.s, 8);
        mbar_init(&bar.wd, 8);
        mbar_init(&bar.upd, 1);
        mbar_init(&bar.qs, 1);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, 8);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
        bar.abort = 0;
    }
    if (warp == 0) tmem_alloc(&bar.tmem, 512);
    if (blockIdx.x == 0) lin::check_seqlens(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const int64_t items = item_count(o);
    int loads = 0;  // stages loaded by the TMA warp (for the way out of an abort)

    if (warp == 12) {
        // --------------------------------------------------------- TMA warp
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = item_at(o, i);
            const Call& c = o.calls.c[t.call];
            const int blocks = c.da / 64;
            for (int k = 0; k < t.chunks; ++k, ++g) {
                const uint32_t st = g & 1;
                if (g >= 2 && !wait(&bar.done[st], ((g - 2) >> 1) & 1, p.err, abort)) {
                    ok = false;
                    break;
                }
                int t0;
                int len;
                chunk_at(t, c.reverse, k, t0, len);
                if (lane == 0) {
                    uint8_t* s = sm + st * kStage;
                    mbar_expect_tx(&bar.full[st], blocks * 32768 + 16384);
                    for (int b = 0; b < blocks; ++b) {
                        tma_load_3d(s + kSX + b * 16384, &o.x[t.call], 64 * b, t.h, t0,
                                    &bar.full[st]);
                        tma_load_3d(s + kSY + b * 16384, &o.y[t.call], 64 * b, t.h, t0,
                                    &bar.full[st]);
                    }
                    tma_load_3d(s + kSW, &o.w[t.call], 64 * t.half, t.h, t0, &bar.full[st]);
                }
                loads = (int)g + 1;
            }
        }
    } else if (warp == 13) {
        // --------------------------------------------------------- MMA warp
        constexpr uint32_t id_sc = idesc_bf16(128, 128, false, false);  // X Y^T
        constexpr uint32_t id_aw = idesc_bf16(128, 64, false, true);    // A W, X S
        constexpr uint32_t id_up = idesc_bf16(128, 64, true, true);     // Y^T W
        const uint64_t dWd = sdesc_sw128(sbase + kSWd, 0, 1024);
        const uint64_t dS = sdesc_sw128(sbase + kSS, 0, 1024);
        // of stage 0; stage 1 is kStage bytes on
        const uint64_t dX = sdesc_sw128(sbase + kSX, 0, 1024);
        const uint64_t dYk = sdesc_sw128(sbase + kSY, 0, 1024);
        const uint64_t dYm = sdesc_sw128(sbase + kSY, 16384, 1024);
        const uint64_t dW = sdesc_sw128(sbase + kSW, 0, 1024);
        const uint32_t lead = lane == 0;
        const uint32_t tm = uniform(tmem);
        // chunks ahead of the current one: where the walk of X Y^T stands
        int64_t next_i = blockIdx.x;
        uint32_t next_left = 0, next_blocks = 0;
        uint32_t gn = 0;
        auto issue_sc = [&]() -> bool {  // X Y^T of chunk gn, if there is one
            while (next_left == 0) {
                if (next_i >= items) return true;
                const Item t = item_at(o, next_i);
                next_i += gridDim.x;
                next_left = uniform(t.chunks);
                next_blocks = uniform(o.calls.c[t.call].da / 64);
            }
            const uint32_t st = gn & 1;
            if (!wait(&bar.full[st], (gn >> 1) & 1, p.err, abort)) return false;
            tc_fence_after();
            uint64_t x = dX + (st * kStage >> 4), y = dYk + (st * kStage >> 4);
            for (uint32_t b = 0; b < next_blocks; ++b, x += 16384 >> 4, y += 16384 >> 4)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_ss(tm + kTA + 128 * st, x + (ks * 32 >> 4), y + (ks * 32 >> 4), id_sc,
                           b > 0 || ks > 0, lead);
            commit(&bar.sc[st], lead);
            --next_left;
            ++gn;
            return true;
        };
        uint32_t g = 0;
        bool ok = issue_sc();
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = item_at(o, i);
            const uint32_t blocks = uniform(o.calls.c[t.call].da / 64);
            const uint32_t chunks = uniform(t.chunks);
            for (uint32_t k = 0; k < chunks; ++k, ++g) {
                const uint32_t st = g & 1, ph = (g >> 1) & 1;
                const uint32_t stage = st * kStage >> 4;
                ok = wait(&bar.s, g & 1, p.err, abort) && wait(&bar.wd, g & 1, p.err, abort);
                if (!ok) break;
                tc_fence_after();
                // S += Y^T Wd: 128 tokens in 8 steps, hi and lo (da = 64: the second 64 lanes
                // take whatever the block's second half holds and are never read)
#pragma unroll 4
                for (uint32_t ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (uint32_t part = 0; part < 2; ++part)
                        mma_ss(tm + kTS, dYm + stage + (ks * 2048 >> 4),
                               dWd + ((part * 16384 + ks * 2048) >> 4), id_up, 1, lead);
                commit(&bar.upd, lead);
                // X S
                for (uint32_t b = 0; b < blocks; ++b)
#pragma unroll
                    for (uint32_t ks = 0; ks < 4; ++ks)
#pragma unroll
                        for (uint32_t part = 0; part < 2; ++part)
                            mma_ss(tm + kTO2 + 64 * st, dX + stage + ((b * 16384 + ks * 32) >> 4),
                                   dS + ((part * 16384 + (4 * b + ks) * 2048) >> 4), id_aw,
                                   b + ks + part > 0, lead);
                commit(&bar.qs, lead);
                if (!(ok = issue_sc())) break;
                ok = wait(&bar.a[st], ph, p.err, abort) &&
                     (g == 0 || wait(&bar.o_free, (g - 1) & 1, p.err, abort));
                if (!ok) break;
                tc_fence_after();
                // A W: A's 16-token steps are 8 columns of hi and 8 of lo
#pragma unroll 4
                for (uint32_t ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (uint32_t part = 0; part < 2; ++part)
                        mma_ts(tm + kTO1, tm + kTA + 128 * st + 16 * ks + 8 * part,
                               dW + stage + (ks * 2048 >> 4), id_aw, ks + part > 0, lead);
                commit(&bar.o_full, lead);
                commit(&bar.done[st], lead);
            }
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ A warps
        const int q = warp;
        const uint32_t lb = static_cast<uint32_t>(32 * q) << 16;
        float* col = reinterpret_cast<float*>(sm + kSCol);
        float* diag = reinterpret_cast<float*>(sm + kSDiag);
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = item_at(o, i);
            const int rev = o.calls.c[t.call].reverse;
            const bool dots = o.calls.c[t.call].dot != nullptr;
            int t0;
            int len;
            float e[4];
            if (t.chunks) {
                chunk_at(t, rev, 0, t0, len);
                load_decays(p, t0, len, t.h, lane, e);
            }
            for (int k = 0; k < t.chunks; ++k, ++g) {
                const uint32_t st = g & 1;
                const Sums s = sums<true>(e, q, lane);
                const int this_len = len;
                col[128 * st + 32 * q + lane] = ex2f(rev ? s.P : s.U);
                if (k + 1 < t.chunks) {
                    chunk_at(t, rev, k + 1, t0, len);
                    load_decays(p, t0, len, t.h, lane, e);
                }
                // all four warps are past the previous chunk and their column factors written
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.col[st]);
                if (!wait(&bar.col[st], (g >> 1) & 1, p.err, abort) ||
                    !wait(&bar.sc[st], (g >> 1) & 1, p.err, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = tmem + lb + kTA + 128 * st;
                float to_block = rev ? s.U : s.P;  // log2 decay between the row and block j
#pragma unroll 1
                for (int n = 0; n < 4; ++n) {  // blocks at distance n from the diagonal
                    const int j = rev ? q + n : q - n, z = rev ? q - n : q + n;
                    if (n > 0 && z >= 0 && z < 4) {  // outside the triangle
                        uint32_t zero[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) zero[c] = 0u;
                        tmem_st32(at + 32 * z, zero);
                    }
                    if (j < 0 || j > 3) continue;
                    float v[32];
                    tmem_ld32(at + 32 * j, v);
                    landed(v);
                    if (n == 0) {
                        // columns of the triangle that are tokens of the segment
                        uint32_t in = rev ? ~((1u << lane) - 1u) : (2u << lane) - 1u;
                        if (rev && this_len - 32 * q < 32)
                            in &= this_len > 32 * q ? (1u << (this_len - 32 * q)) - 1u : 0u;
                        if (dots) {
                            float own = 0.f;
#pragma unroll
                            for (int c = 0; c < 32; ++c) own = c == lane ? v[c] : own;
                            diag[128 * (g % 3) + 32 * q + lane] = own;
                            in &= ~(1u << lane);
                        }
                        const float ph = rev ? -s.P : s.P, pl = rev ? -s.Plo : s.Plo;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float x = (ph - __shfl_sync(0xffffffffu, ph, c)) +
                                            (pl - __shfl_sync(0xffffffffu, pl, c));
                            v[c] = in & (1u << c) ? v[c] * ex2f(x) : 0.f;
                        }
                    } else {
                        const float rf = ex2f(to_block);
                        to_block += pick(s.B, j);
                        const float4* cf = reinterpret_cast<const float4*>(col + 128 * st + 32 * j);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float4 f = cf[c];
                            v[4 * c] *= rf * f.x;
                            v[4 * c + 1] *= rf * f.y;
                            v[4 * c + 2] *= rf * f.z;
                            v[4 * c + 3] *= rf * f.w;
                        }
                        if (rev && this_len - 32 * j < 32)
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (32 * j + c >= this_len) v[c] = 0.f;
                    }
                    uint32_t u[32];  // each 16-token step: 8 columns of hi, 8 of lo
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const int k2 = 16 * (c >> 3) + (c & 7);
                        u[k2] = pack_bf16x2(v[2 * c], v[2 * c + 1]);
                        u[k2 + 8] =
                            pack_bf16x2(v[2 * c] - __uint_as_float(u[k2] << 16),
                                        v[2 * c + 1] - __uint_as_float(u[k2] & 0xffff0000u));
                    }
                    tmem_st32(at + 32 * j, u);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.a[st]);
            }
        }
    } else {
        // --------------------------------------- state, decayed W and outputs
        const int q = warp & 3, wg = (warp - 4) >> 2;
        const int row = 32 * q + lane;  // token, or state row
        const uint32_t lb = static_cast<uint32_t>(32 * q) << 16;
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = item_at(o, i);
            const Call& c = o.calls.c[t.call];
            const int rev = c.reverse;
            const int64_t E = (int64_t)c.da * c.db;
            const int64_t rs = c.tr ? 1 : c.db, cs = c.tr ? c.da : 1;
            const int64_t mine = (int64_t)row * rs + (int64_t)(64 * t.half + 32 * wg) * cs;
            const int64_t seq = ((int64_t)t.sg.n * p.H + t.h) * E + mine;
            const bool sv = row < c.da;  // this lane holds a state row
            if (!t.live) {
                // an empty sequence owns its first slot: its final state is its initial one
                if (c.S_out && t.sg.count == 0 && t.sg.s == 0 && t.half * 64 < c.db && sv)
                    for (int x = 0; x < 32; ++x)
                        c.S_out[seq + x * cs] = c.edge ? c.edge[seq + x * cs] : 0.f;
                continue;
            }
            const float* from =
                t.sg.count > 1 ? c.seg + ((int64_t)t.slot * p.H + t.h) * E + mine
                               : c.edge ? c.edge + seq : nullptr;
            int t0, len;
            float e[4];
            chunk_at(t, rev, 0, t0, len);
            load_decays(p, t0, len, t.h, lane, e);
            {
                // the segment's edge state into TMEM, once the last segment's is done with
                float S[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) S[x] = 0.f;
                if (from && sv) {
                    if (c.tr) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) S[x] = __ldcg(from + x * cs);
                    } else {
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const float4 f = __ldcg(reinterpret_cast<const float4*>(from) + x);
                            S[4 * x] = f.x;
                            S[4 * x + 1] = f.y;
                            S[4 * x + 2] = f.z;
                            S[4 * x + 3] = f.w;
                        }
                    }
                }
                if (g > 0 && !wait(&bar.upd, (g - 1) & 1, p.err, abort)) { ok = false; break; }
                tc_fence_after();
                uint32_t u[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(S[x]);
                tmem_st32(tmem + lb + kTS + 32 * wg, u);
                tmem_st_wait();
            }
            int t0_prev = 0, len_prev = 0;
            float rowf_prev = 0.f;
            // step k: the state's copy and the decayed W of chunk k, then the outputs of chunk
            // k - 1 while the tensor cores work on chunk k
#pragma unroll 1
            for (int k = 0; k <= t.chunks; ++k) {
                const int t0_now = t0, len_now = len;
                float rowf = 0.f;
                if (k < t.chunks) {
                    const uint32_t st = g & 1;
                    const Sums s = sums<false>(e, q, lane);
                    const float head = s.P + before(s, q), tail = s.U + after(s, q);
                    rowf = ex2f(rev ? tail : head);
                    const float wf = row < len ? ex2f(rev ? head : tail) : 0.f;
                    const float all = ex2f((s.B[0] + s.B[1]) + (s.B[2] + s.B[3]));
                    if (k + 1 < t.chunks) {
                        chunk_at(t, rev, k + 1, t0, len);
                        load_decays(p, t0, len, t.h, lane, e);
                    }
                    // the last update of the state, the last read of its copy and of the decayed
                    // W's buffer are complete
                    if (g > 0 && (!wait(&bar.upd, (g - 1) & 1, p.err, abort) ||
                                  !wait(&bar.qs, (g - 1) & 1, p.err, abort))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    uint8_t* sr = sm + kSS + row * 128;
#pragma unroll 1
                    for (int b = 0; b < 2; ++b) {
                        float S[16];
                        tmem_ld16(tmem + lb + kTS + 32 * wg + 16 * b, S);
                        landed(S);
                        if (sv)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                float v[8];
#pragma unroll
                                for (int y = 0; y < 8; ++y) v[y] = S[8 * x + y];
                                uint4 hi, lo;
                                pk8_hilo(v, hi, lo);
                                const uint32_t at = ((4 * wg + 2 * b + x) ^ (row & 7)) << 4;
                                *reinterpret_cast<uint4*>(sr + at) = hi;
                                *reinterpret_cast<uint4*>(sr + 16384 + at) = lo;
                            }
                        uint32_t u[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(S[x] * all);
                        tmem_st16(tmem + lb + kTS + 32 * wg + 16 * b, u);
                    }
                    tmem_st_wait();
                    fence_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.s);

                    if (!wait(&bar.full[st], (g >> 1) & 1, p.err, abort)) { ok = false; break; }
                    uint8_t* stage = sm + st * kStage;
                    uint8_t* wr = stage + kSW + row * 128;
                    uint8_t* wd = sm + kSWd + row * 128;
                    const bool dead = row >= len_now;
#pragma unroll 2
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t at = ((4 * wg + x) ^ (row & 7)) << 4;
                        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
                        if (!dead) {
                            float v[8];
                            ld8(wr + at, v);
#pragma unroll
                            for (int y = 0; y < 8; ++y) v[y] *= wf;
                            pk8_hilo(v, hi, lo);
                        } else {
                            // rows past the segment hold another sequence's tokens (or zeros):
                            // they must not reach a product even as 0 * inf
                            *reinterpret_cast<uint4*>(wr + at) = hi;
                        }
                        *reinterpret_cast<uint4*>(wd + at) = hi;
                        *reinterpret_cast<uint4*>(wd + 16384 + at) = lo;
                    }
                    if (dead && 64 * wg < c.da) {
                        uint4* yr = reinterpret_cast<uint4*>(stage + kSY + wg * 16384 + row * 128);
#pragma unroll 1
                        for (int x = 0; x < 8; ++x) yr[x] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.wd);
                    ++g;
                }
                if (k > 0) {
                    // Outputs of chunk k - 1: rowf (X S) + A W.  Where their dot products with
                    // another row are wanted, A W comes without the diagonal's term
                    // x_r . y_r w_r, which is added here in fp32 and left out of the dot: it is
                    // the same number in both of the decay's gradient's sums, where under strong
                    // decays everything else is far below its rounding.
                    const uint32_t gg = k < t.chunks ? g - 2 : g - 1;
                    if (!wait(&bar.o_full, gg & 1, p.err, abort)) { ok = false; break; }
                    tc_fence_after();
                    const int tr = t0_prev + row;
                    const int off = t.h * c.db + 64 * t.half + 32 * wg;
                    const bool in = row < len_prev;
                    uint8_t* out = static_cast<uint8_t*>(c.out) +
                                   ((int64_t)tr * p.H * c.db + off) * 2;
                    float acc = 0.f;
#pragma unroll 1
                    for (int b = 0; b < 2; ++b) {
                        float o1[16], o2[16];
                        tmem_ld16(tmem + lb + kTO1 + 32 * wg + 16 * b, o1);
                        tmem_ld16(tmem + lb + kTO2 + 64 * (gg & 1) + 32 * wg + 16 * b, o2);
                        landed(o1);
                        landed(o2);
#pragma unroll
                        for (int x = 0; x < 16; ++x) o1[x] = fmaf(rowf_prev, o2[x], o1[x]);
                        if (in && c.dot) {
                            const uint8_t* dr = static_cast<const uint8_t*>(c.dot) +
                                                ((int64_t)tr * c.dot_ld + off) * 2 + 32 * b;
                            const uint8_t* wr = static_cast<const uint8_t*>(c.w) +
                                                ((int64_t)tr * c.w_ld + off) * 2 + 32 * b;
                            const float dg =
                                reinterpret_cast<const float*>(sm + kSDiag)[128 * (gg % 3) + row];
#pragma unroll
                            for (int h8 = 0; h8 < 2; ++h8) {
                                float d[8], w[8];
                                ld8(dr + 16 * h8, d);
                                ld8(wr + 16 * h8, w);
#pragma unroll
                                for (int x = 0; x < 8; ++x) {
                                    acc = fmaf(o1[8 * h8 + x], d[x], acc);
                                    o1[8 * h8 + x] = fmaf(dg, w[x], o1[8 * h8 + x]);
                                }
                            }
                        }
                        if (in) {
                            uint4 u[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                u[x] = make_uint4(pack_bf16x2(o1[8 * x], o1[8 * x + 1]),
                                                  pack_bf16x2(o1[8 * x + 2], o1[8 * x + 3]),
                                                  pack_bf16x2(o1[8 * x + 4], o1[8 * x + 5]),
                                                  pack_bf16x2(o1[8 * x + 6], o1[8 * x + 7]));
                            if (o.wide_store) {
                                st_global_32(out + 32 * b, u[0], u[1]);
                            } else {
                                reinterpret_cast<uint4*>(out)[2 * b] = u[0];
                                reinterpret_cast<uint4*>(out)[2 * b + 1] = u[1];
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.o_free);
                    if (in && c.dot)
                        c.dots[((int64_t)(2 * t.half + wg) * p.T + tr) * p.H + t.h] = acc;
                }
                t0_prev = t0_now;
                len_prev = len_now;
                rowf_prev = rowf;
            }
            if (!ok) break;
            const bool last = rev ? t.sg.s == 0 : t.sg.s == t.sg.count - 1;
            if (last && c.S_out) {  // (the chunk's outputs are complete, so its update is too)
                float S[32];
                tmem_ld32(tmem + lb + kTS + 32 * wg, S);
                landed(S);
                if (sv)
#pragma unroll
                    for (int x = 0; x < 32; ++x) c.S_out[seq + x * cs] = S[x];
            }
        }
    }

    __syncthreads();
    if (bar.abort) {
        // let copies and MMAs still in flight land before leaving
        if (warp == 12)
            for (int x = max(loads - 2, 0); x < loads; ++x)
                mbar_wait(&bar.full[x & 1], (x >> 1) & 1, nullptr);
        if (tid == 13 * 32) {
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, nullptr);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// --------------------------------------------------------- segment sums --
// sum_i e^{G_end - G_i} y_i w_i^T over a segment [reversed: e^{G_i} from its start].  The order
// of a sum is free, so the chunks run away from the edge the weights refer to, the decay between
// the edge and the chunk carried along, and the accumulator in TMEM is never rescaled.  W is
// decayed in place (hi over W itself, lo beside it), so two stages of all operands fit.  Bound by
// reading Y and W.
constexpr int kSumThreads = 384;
constexpr uint32_t kUY = 0, kUW = 32768, kULo = 65536, kUStage = 98304;  // two stages
constexpr uint32_t kUBar = 2 * kUStage;
constexpr uint32_t kSumSmem = kUBar + 256;

struct SumBars {
    uint64_t full[2], done[2], wd[2], drain;
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
    static_assert(kC == 128, "a chunk is the 128 lanes of a TMEM tile");
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.done[i], 1);
            mbar_init(&bar.wd[i], 8);
        }
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
        bar.abort = 0;
    }
    if (warp == 0) tmem_alloc(&bar.tmem, 128);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const int64_t items = item_count(o);
    // an item whose sum no edge needs: the last segment of a walk
    auto skip = [&](const Item& t) {
        const int rev = o.calls.c[t.call].reverse;
        return !t.live || (rev ? t.sg.s == 0 : t.sg.s == t.sg.count - 1);
    };
    int loads = 0;

    if (warp == 0) {
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = item_at(o, i);
            if (skip(t)) continue;
            const Call& c = o.calls.c[t.call];
            for (int k = 0; k < t.chunks; ++k, ++g) {
                const uint32_t st = g & 1;
                if (g >= 2 && !wait(&bar.done[st], ((g - 2) >> 1) & 1, p.err, abort)) {
                    ok = false;
                    break;
                }
                int t0;
                int len;
                chunk_at(t, !c.reverse, k, t0, len);
                if (lane == 0) {
                    uint8_t* s = sm + st * kUStage;
                    mbar_expect_tx(&bar.full[st], (c.da + c.db) / 64 * 16384);
                    for (int b = 0; b < c.da / 64; ++b)
                        tma_load_3d(s + kUY + b * 16384, &o.y[t.call], 64 * b, t.h, t0,
                                    &bar.full[st]);
                    for (int b = 0; b < c.db / 64; ++b)
                        tma_load_3d(s + kUW + b * 16384, &o.w[t.call], 64 * b, t.h, t0,
                                    &bar.full[st]);
                }
                loads = (int)g + 1;
            }
        }
    } else if (warp == 1) {
        const uint32_t lead = lane == 0;
        const uint32_t tm = uniform(tmem);
        const uint64_t dY = sdesc_sw128(sbase + kUY, 16384, 1024);
        const uint64_t dHi = sdesc_sw128(sbase + kUW, 16384, 1024);
        const uint64_t dLo = sdesc_sw128(sbase + kULo, 16384, 1024);
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = item_at(o, i);
            if (skip(t)) continue;
            const Call& c = o.calls.c[t.call];
            const uint32_t id = uniform(idesc_bf16(128, 64, true, true) +
                                        (c.db == 128 ? (64u >> 3) << 17 : 0u));  // N = db
            const uint32_t chunks = uniform(t.chunks);
            for (uint32_t k = 0; k < chunks; ++k, ++g) {
                const uint32_t st = g & 1;
                if (!wait(&bar.wd[st], (g >> 1) & 1, p.err, abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t stage = st * kUStage >> 4;
#pragma unroll 4
                for (uint32_t ks = 0; ks < 8; ++ks) {
                    const uint32_t at = stage + (ks * 2048 >> 4);
                    mma_ss(tm, dY + at, dHi + at, id, k + ks > 0, lead);
                    mma_ss(tm, dY + at, dLo + at, id, 1, lead);
                }
                commit(&bar.done[st], lead);
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3, wg = (warp - 4) >> 2;
        const int row = 32 * q + lane;
        const uint32_t lb = static_cast<uint32_t>(32 * q) << 16;
        uint32_t g = 0;
        bool ok = true;
        for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item t = item_at(o, i);
            if (skip(t)) continue;
            const Call& c = o.calls.c[t.call];
            const int rev = c.reverse;
            float between = 0.f;  // log2 decay between the edge and the chunk
            int t0;
            int len;
            float e[4];
            chunk_at(t, !rev, 0, t0, len);
            load_decays(p, t0, len, t.h, lane, e);
            for (int k = 0; k < t.chunks; ++k, ++g) {
                const uint32_t st = g & 1;
                const Sums s = sums<false>(e, q, lane);
                const float head = s.P + before(s, q), tail = s.U + after(s, q);
                const float wf = ex2f((rev ? head : tail) + between);
                between += (s.B[0] + s.B[1]) + (s.B[2] + s.B[3]);
                const int len_now = len;
                if (k + 1 < t.chunks) {
                    chunk_at(t, !rev, k + 1, t0, len);
                    load_decays(p, t0, len, t.h, lane, e);
                }
                if (!wait(&bar.full[st], (g >> 1) & 1, p.err, abort)) { ok = false; break; }
                uint8_t* stage = sm + st * kUStage;
                const bool dead = row >= len_now;
                if (64 * wg < c.db) {
                    uint8_t* wr = stage + kUW + wg * 16384 + row * 128;
                    uint8_t* lr = stage + kULo + wg * 16384 + row * 128;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const uint32_t at = (x ^ (row & 7)) << 4;
                        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
                        if (!dead) {
                            float v[8];
                            ld8(wr + at, v);
#pragma unroll
                            for (int y = 0; y < 8; ++y) v[y] *= wf;
                            pk8_hilo(v, hi, lo);
                        }
                        *reinterpret_cast<uint4*>(wr + at) = hi;
                        *reinterpret_cast<uint4*>(lr + at) = lo;
                    }
                }
                if (dead && 64 * wg < c.da) {
                    uint4* yr = reinterpret_cast<uint4*>(stage + kUY + wg * 16384 + row * 128);
#pragma unroll
                    for (int x = 0; x < 8; ++x) yr[x] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.wd[st]);
            }
            if (!ok) break;
            // the accumulator is complete with the item's last chunk; the next item's first MMA
            // follows this warp's next arrival
            const uint32_t gl = g - 1;
            if (!wait(&bar.done[gl & 1], (gl >> 1) & 1, p.err, abort)) { ok = false; break; }
            tc_fence_after();
            const int64_t at = (((int64_t)t.slot * p.H + t.h) * c.da + row) * c.db + 64 * wg;
            if (64 * wg < c.db) {
                float* to = const_cast<float*>(c.seg) + at;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float v[32];
                    tmem_ld32(tmem + lb + 64 * wg + 32 * b, v);
                    landed(v);
                    if (row < c.da)
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            reinterpret_cast<float4*>(to)[8 * b + x] =
                                make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                }
            }
            tc_fence_before();
            if (warp == 4 && lane == 0)
                dec[((int64_t)rev * o.slots + t.slot) * p.H + t.h] = between;
        }
    }

    __syncthreads();
    if (bar.abort) {
        if (warp == 0)
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
        tmem_dealloc(tmem, 128);
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

int sm_count() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 1;
}

cudaError_t fill(OutParams& o, const Problem& p, const lin::Calls& calls, int n, int64_t slots,
                 bool out) {
    o.p = p;
    o.calls = calls;
    o.n_calls = n;
    o.slots = slots;
    o.wide_store = 1;
    for (int i = 0; i < n; ++i) {
        const Call& c = calls.c[i];
        if (out && c.db == 128) o.halves = 2;
        if (reinterpret_cast<uintptr_t>(c.out) & 31) o.wide_store = 0;
        if (p.T == 0) continue;
        if ((out && !make_map(&o.x[i], c.x, p.T, p.H, c.da, c.x_ld)) ||
            !make_map(&o.y[i], c.y, p.T, p.H, c.da, c.y_ld) ||
            !make_map(&o.w[i], c.w, p.T, p.H, c.db, c.w_ld))
            return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_outputs(const Problem& p, const lin::Calls& calls, int n, int64_t slots,
                           const char* name, cudaStream_t s) {
    OutParams o{};
    o.halves = 1;
    if (cudaError_t e = fill(o, p, calls, n, slots, true)) return e;
    if (cudaError_t e = cudaFuncSetAttribute(
            out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kOutSmem))
        return e;
    const int64_t items = slots * p.H * n * o.halves, sms = sm_count();
    ProfScope prof(name, s);
    out_kernel<<<(unsigned)(items < sms ? items : sms), kThreads, kOutSmem, s>>>(o);
    return cudaGetLastError();
}

cudaError_t launch_sums(const Problem& p, const lin::Calls& calls, int n, int64_t slots,
                        float* dec, const char* name, cudaStream_t s) {
    OutParams o{};
    o.halves = 1;
    if (cudaError_t e = fill(o, p, calls, n, slots, false)) return e;
    if (cudaError_t e = cudaFuncSetAttribute(
            sum_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSumSmem))
        return e;
    const int64_t items = slots * p.H * n, sms = sm_count();
    ProfScope prof(name, s);
    sum_kernel<<<(unsigned)(items < sms ? items : sms), kSumThreads, kSumSmem, s>>>(o, dec);
    return cudaGetLastError();
}

}  // namespace lintc
}  // namespace kda
