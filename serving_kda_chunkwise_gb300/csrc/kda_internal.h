// kda_internal.h -- host-side launchers shared between the C ABI (api.cu) and the
// kernel translation units.  Not part of the public interface (that is include/kda.h).
#pragma once

#include <cuda_runtime.h>

#include "kda.h"
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct FwdArgs {
    const void *q, *k, *v, *beta, *z;
    const float* A_log;
    float g_min;
    const float* S0;
    float* S_out;
    const int32_t* cu_seqlens;
    int N;
    int64_t T_total;
    int H, dk, dv;
    int io_bf16;  // 1: bf16 I/O, 0: fp32 I/O
    int gate_kind;  // 0: g_min Sigmoid(e^A z); 1: -e^A Softplus(z)
    void* o;              // may be nullptr on the tensor-core path (no output stored)
    void* workspace;
    size_t ws_bytes;
    unsigned* dev_err;
    cudaStream_t stream;
    // tensor-core path only, for a backward pass (nullptr otherwise; o must then be nullptr):
    // the backward's image blocks [chunks][H] in the order of the chunk offsets
    // (bwd_tc_layout.cuh), which receive S_0, Vt and N of every chunk; selects the two-launch
    // form, which also leaves every (chunk, head) package in the workspace
    void* bimg;
    // two-launch form, optional: recorded on `stream` once the intra stage is enqueued (the
    // backward starts its gradient chain on a second stream from there)
    cudaEvent_t after_intra;
};

struct BwdArgs {
    const void *q, *k, *v, *beta, *z, *dout;
    const float* A_log;
    float g_min;
    const float* S0;
    const float* dS_out;
    const int32_t* cu_seqlens;
    int N;
    int64_t T_total;
    int H, dk, dv;
    int io_bf16;
    void *dq, *dk_, *dv_, *dbeta, *dz;
    float* dA_log;
    float* dS0;
    void* workspace;
    unsigned* dev_err;
    cudaStream_t stream;
};

// Gradients of the forward (bwd.cu): token-level reverse mode on CUDA cores.
size_t bwd_workspace_size_public(int64_t T_total, int N, int H, int dk, int dv);
cudaError_t launch_bwd(const BwdArgs& a);

// A bounded wait that runs out (selftest.cu): sets the timeout bit of the error word.
cudaError_t launch_selftest_timeout(uint64_t limit_ns, unsigned* err, cudaStream_t stream);

// K1: elementwise gate.
cudaError_t launch_gate(const void* z, int z_bf16, const float* A_log, float g_min, float* g_out,
                        int64_t n_tokens, int H, int dk, cudaStream_t stream);

// K4: one decode token per sequence, state updated in place.
cudaError_t launch_decode(const void* q, const void* k, const void* v, const void* beta,
                          const void* z, const float* A_log, float g_min, float* S, int N, int H,
                          int dk, int dv, int io_bf16, void* o, cudaStream_t stream);

// K4 with the gated output step of "Gated MLA" fused: writes y instead of o.
cudaError_t launch_decode_gated(const void* q, const void* k, const void* v, const void* beta,
                                const void* z, const float* A_log, float g_min, float* S, int N,
                                int H, int dk, int dv, int io_bf16, const void* gate,
                                const float* norm_w, float eps, void* y, cudaStream_t stream);

// The gated output step alone: rows of dv channels (one per token and head).
cudaError_t launch_output_gate(const void* o, const void* gate, const float* norm_w, float eps,
                               void* y, int64_t n_rows, int dv, int io_bf16,
                               cudaStream_t stream);

// Quantile-balancing bias update of the expert router (qb.cu).
size_t qb_workspace_size(int64_t m, int n);
cudaError_t launch_quantile_balance(const float* s, const float* b, int64_t m, int n, int k,
                                    float* b_new, float* bhat, float* alpha, void* workspace,
                                    cudaStream_t stream);

// Linear attention with one decay per head (linear.cu; the tensor-core outputs linear_tc.cu).
struct LinearArgs {
    const void *q, *k, *v;
    int64_t q_ld, k_ld, v_ld;
    const float* g;
    int g_per_token;
    const float* S0;
    float* S_out;  // backward: unused
    const int32_t* cu_seqlens;
    int N;
    int64_t T_total;
    int H, dk, dv;
    int io_bf16;
    void* o;
    // backward only
    const void* dout;
    int64_t dout_ld;
    const float* dS_out;
    void *dq, *dk_, *dv_;
    float *dg, *dS0;
    void* workspace;
    unsigned* dev_err;
    cudaStream_t stream;
};
size_t linear_fwd_workspace_size(int64_t T_total, int N, int H, int dk, int dv, int io_bf16);
size_t linear_bwd_workspace_size(int64_t T_total, int N, int H, int dk, int dv, int io_bf16);
cudaError_t launch_linear_fwd(const LinearArgs& a);
cudaError_t launch_linear_bwd(const LinearArgs& a);
cudaError_t launch_linear_decode(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                 const void* v, int64_t v_ld, const float* g, int g_per_token,
                                 float* S, const int32_t* slots, int n_slots, int N, int H, int dk,
                                 int dv, int io_bf16, void* o, unsigned* dev_err,
                                 cudaStream_t stream);

// Norm of the query and key heads with the position rotation (qk_norm.cu).
struct QkNormArgs {
    const void *q, *k;
    int64_t q_ld, k_ld;
    const void *dyq, *dyk;  // backward only
    const float *wq, *wk;
    float eps;
    const float* cos_sin;
    int64_t n_pos;
    const int32_t* positions;
    int rot_dim, interleaved;
    void *q_out, *k_out;  // backward: dq, dk
    float *dwq, *dwk;     // backward only
    int64_t T;
    int Hq, Hk, d;
    int io_bf16;
    void* workspace;
    unsigned* dev_err;
    cudaStream_t stream;
};
size_t qk_norm_bwd_workspace_size(int d);
cudaError_t launch_qk_norm(const QkNormArgs& a);
cudaError_t launch_qk_norm_bwd(const QkNormArgs& a);

// The gated recurrence of single channels (recurrence.cu).
struct RecurrenceArgs {
    const void *x, *z, *i;                       // io_dt, or codes when packed
    int64_t x_ld, z_ld, i_ld;
    const int8_t *x_exps, *z_exps, *i_exps;      // packed inputs only
    int packed;
    const float* A_log;
    float g_min;
    const float* h0;
    float* h_out;  // backward: unused
    const int32_t* cu_seqlens;
    int N;
    int64_t T_total;
    int D;
    int io_bf16;
    void* y;       // forward: nullptr when only the edges are wanted
    float* edges;  // forward: written, or nullptr; backward: read, or nullptr
    // backward only
    const void* dy;
    int64_t dy_ld;
    const float* dh_out;
    void *dx, *dz, *di;
    float *dA_log, *dh0;
    void* workspace;
    unsigned* dev_err;
    cudaStream_t stream;
};
size_t recurrence_fwd_workspace_size(int64_t T_total, int N, int D);
size_t recurrence_bwd_workspace_size(int64_t T_total, int N, int D);
cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a);
cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a);
cudaError_t launch_recurrence_step(const void* x, int64_t x_ld, const void* z, int64_t z_ld,
                                   const void* i, int64_t i_ld, const float* A_log, float g_min,
                                   float* h, const int32_t* slots, int n_slots, int N, int D,
                                   int io_bf16, void* y, unsigned* dev_err, cudaStream_t stream);

// Activations in 8 bits (checkpoint.cu).
cudaError_t launch_checkpoint_pack(const void* x, int64_t x_ld, int64_t T, int D, int io_bf16,
                                   int8_t* codes, int8_t* exps, cudaStream_t stream);
cudaError_t launch_checkpoint_unpack(const int8_t* codes, const int8_t* exps, int64_t T, int D,
                                     int io_bf16, void* x, cudaStream_t stream);

// Norms before and after a block, with its gate and residual (block_norm.cu).
struct BlockNormArgs {
    const void *y, *gate, *r;  // r: the residual before the block (forward) or after it (backward)
    const float *scale, *w_post, *w_pre;
    int post_norm;
    float eps;
    void *r_out, *x_out;       // forward only
    const void *dx, *dr;       // backward only, as the rest
    void *dr_in, *dy, *dgate;
    float *dscale, *dw_post, *dw_pre;
    int64_t T;
    int D;
    int io_bf16, r_bf16;
    void* workspace;
    unsigned* dev_err;  // backward only
    cudaStream_t stream;
};
constexpr int kMaxBlockNormD = 8192;
size_t block_norm_bwd_workspace_size(int D);
cudaError_t launch_block_norm(const BlockNormArgs& a);
cudaError_t launch_block_norm_bwd(const BlockNormArgs& a);

// Chunked forward on CUDA cores in fp32 (any dtype, dk/dv in {64,128}).
cudaError_t launch_fwd_generic(const FwdArgs& a);

// Chunked forward on tcgen05 tensor cores (bf16 I/O, dk = dv = 128); needs a workspace of
// fwd_tc_workspace_size() bytes.
size_t fwd_tc_workspace_size(int64_t T_total, int N, int H);
cudaError_t launch_fwd_tc(const FwdArgs& a);

// The backward's gradient chain on tcgen05 tensor cores (bwd_chain_tc.cu), bf16 problems:
// from the packages that launch_fwd_tc with bimg set left in `fwd_ws`, the state's gradient
// at every chunk end and dVt into the image blocks `bimg`, and a.dS0.
cudaError_t launch_bwd_chain_tc(const BwdArgs& a, void* fwd_ws, void* bimg, cudaStream_t stream);

// The backward's per-chunk kernels on tcgen05 tensor cores (bwd_item_tc.cu), bf16 problems:
// from the image blocks, every gradient but dS0, plus the [chunks][H] dA_log partials; `mid`
// holds the mid blocks between its two kernels.
cudaError_t launch_bwd_items_tc(const BwdArgs& a, void* fwd_ws, const void* bimg, void* mid,
                                float* dA_item, cudaStream_t stream);

// The argument checks of kda_fwd_chunked except those of the workspace (api.cu): KDA_OK, or
// the failing status with the calling thread's last error set.
kda_status_t check_fwd_args(const void* q, const void* k, const void* v, const void* beta,
                            const void* z, const float* A_log, float g_min, const float* S0,
                            float* S_out, const int32_t* cu_seqlens, int N, int64_t T_total,
                            int H, int dk, int dv, kda_dtype_t io_dt, void* o);

// Records `msg` as the calling thread's last error (see kda_last_error) and returns `s`.
kda_status_t set_last_error(kda_status_t s, const char* msg);

// Kernel timing hooks (profile.cu): no-ops unless kda_profile_begin() is active.
int prof_kernel_begin(const char* name, cudaStream_t s);
void prof_kernel_end(int ev, cudaStream_t s);

struct ProfScope {
    int ev;
    cudaStream_t s;
    ProfScope(const char* name, cudaStream_t stream) : ev(prof_kernel_begin(name, stream)), s(stream) {}
    ~ProfScope() { prof_kernel_end(ev, s); }
    ProfScope(const ProfScope&) = delete;
    ProfScope& operator=(const ProfScope&) = delete;
};

}  // namespace kda
