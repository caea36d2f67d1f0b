// api.cu -- the C ABI of libkda.so (declared in include/kda.h): argument checks,
// kernel selection and the device error word.  No entry point allocates device memory.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_internal.h"

namespace {

__device__ unsigned g_device_error = 0u;

thread_local std::string t_last_error;

kda_status_t fail(kda_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kda_status_t fail(kda_status_t s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    t_last_error = buf;
    return s;
}

kda_status_t cuda_fail(cudaError_t e, const char* where) {
    return fail(KDA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define KDA_REQUIRE(cond, ...)                                   \
    do {                                                         \
        if (!(cond)) return fail(KDA_ERR_INVALID_ARG, __VA_ARGS__); \
    } while (0)

#define KDA_REQUIRE_PTR(p, name)                                                   \
    do {                                                                           \
        if ((p) == nullptr) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);  \
        if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name); \
    } while (0)

// Arrays of 4-byte values read one by one (so that a slice of a longer one can be passed).
#define KDA_REQUIRE_WORDS(p, name)                                                      \
    do {                                                                                \
        if ((p) == nullptr) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);       \
        if (reinterpret_cast<uintptr_t>(p) & 3u)                                        \
            return fail(KDA_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);         \
    } while (0)

#define KDA_OPTIONAL_PTR(p, name)                                                  \
    do {                                                                           \
        if ((p) != nullptr && !aligned16(p))                                       \
            return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);   \
    } while (0)

// Device address of the error word on the current device (looked up once per device).
unsigned* device_error_ptr() {
    static std::mutex mu;
    static unsigned* cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev] == nullptr) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
        cache[dev] = static_cast<unsigned*>(p);
    }
    return cache[dev];
}

kda_status_t check_dims(int dk, int dv) {
    if (dk <= 0 || dv <= 0) return fail(KDA_ERR_INVALID_ARG, "dk=%d dv=%d must be positive", dk, dv);
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128))
        return fail(KDA_ERR_UNSUPPORTED, "dk=%d dv=%d: only 64 and 128 are supported", dk, dv);
    return KDA_OK;
}

kda_status_t check_gmin(float g_min) {
    if (!(g_min < 0.f) || !std::isfinite(g_min))
        return fail(KDA_ERR_INVALID_ARG, "g_min=%g must be finite and negative", (double)g_min);
    return KDA_OK;
}

}  // namespace

namespace kda {
kda_status_t set_last_error(kda_status_t s, const char* msg) {
    t_last_error = msg;
    return s;
}
}  // namespace kda

extern "C" {

int kda_version(void) { return 400; /* 0.4.0: channel recurrence, 8-bit checkpoints, norms around a block */ }

const char* kda_status_string(kda_status_t s) {
    switch (s) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG";
        case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED";
        case KDA_ERR_CUDA: return "KDA_ERR_CUDA";
        case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT";
        case KDA_ERR_DEVICE: return "KDA_ERR_DEVICE";
    }
    return "KDA_ERR_UNKNOWN";
}

const char* kda_last_error(void) { return t_last_error.c_str(); }

kda_status_t kda_gate(const void* z, kda_dtype_t z_dt, const float* A_log, float g_min,
                      float* g_out, int64_t n_tokens, int H, int dk, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(z_dt == KDA_F32 || z_dt == KDA_BF16, "z_dt=%d is not a kda_dtype_t", (int)z_dt);
    KDA_REQUIRE(n_tokens >= 0, "n_tokens=%lld must be >= 0", (long long)n_tokens);
    KDA_REQUIRE(H > 0, "H=%d must be positive", H);
    KDA_REQUIRE(dk > 0 && dk % 4 == 0, "dk=%d must be a positive multiple of 4", dk);
    if (kda_status_t s = check_gmin(g_min)) return s;
    if (n_tokens == 0) return KDA_OK;
    KDA_REQUIRE_PTR(z, "z");
    KDA_REQUIRE_PTR(A_log, "A_log");
    KDA_REQUIRE_PTR(g_out, "g_out");
    cudaError_t e = kda::launch_gate(z, z_dt == KDA_BF16, A_log, g_min, g_out, n_tokens, H, dk,
                                     reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_gate launch");
    return KDA_OK;
}

// Which forward kernels a problem takes: bf16 I/O the tensor-core path at every head size
// (a 64 runs zero-padded to 128), fp32 I/O the fp32 CUDA-core path.  KDA_FWD_PATH=generic
// in the environment forces the CUDA-core path (the tests use it to cross-check the two).
static bool use_tc_path(int dk, int dv, kda_dtype_t io_dt) {
    if (io_dt != KDA_BF16 || (dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return false;
    const char* env = getenv("KDA_FWD_PATH");
    return !(env && strcmp(env, "generic") == 0);
}

size_t kda_fwd_workspace_size(int64_t T_total, int N, int H, int dk, int dv, kda_dtype_t io_dt) {
    if (T_total < 0 || N < 0 || H <= 0) return 0;
    if (!use_tc_path(dk, dv, io_dt)) return 0;
    return kda::fwd_tc_workspace_size(T_total, N, H);
}

}  // extern "C"

namespace kda {
// The argument checks of kda_fwd_chunked other than the workspace ones (shared with
// kda_fwd_chunked_noalloc, which must report a malformed call before anything else).
kda_status_t check_fwd_args(const void* q, const void* k, const void* v, const void* beta,
                            const void* z, const float* A_log, float g_min, const float* S0,
                            float* S_out, const int32_t* cu_seqlens, int N, int64_t T_total,
                            int H, int dk, int dv, kda_dtype_t io_dt, void* o) {
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(N >= 0, "N=%d must be >= 0", N);
    KDA_REQUIRE(H > 0, "H=%d must be positive", H);
    KDA_REQUIRE(T_total >= 0, "T_total=%lld must be >= 0", (long long)T_total);
    if (kda_status_t s = check_dims(dk, dv)) return s;
    if (kda_status_t s = check_gmin(g_min)) return s;
    if (cu_seqlens == nullptr) {
        KDA_REQUIRE(N > 0 || T_total == 0, "N=0 requires T_total=0");
        KDA_REQUIRE(N == 0 || T_total % N == 0,
                    "without cu_seqlens T_total=%lld must be a multiple of N=%d",
                    (long long)T_total, N);
    }
    KDA_REQUIRE((int64_t)N * H * 4 < (int64_t)1 << 31, "N*H=%lld is too large",
                (long long)N * H);
    if (N == 0) return KDA_OK;
    if (T_total > 0) {
        KDA_REQUIRE_PTR(q, "q");
        KDA_REQUIRE_PTR(k, "k");
        KDA_REQUIRE_PTR(v, "v");
        KDA_REQUIRE_PTR(z, "z");
        KDA_REQUIRE_PTR(o, "o");
        KDA_REQUIRE(beta != nullptr, "beta is NULL");
    }
    KDA_REQUIRE_PTR(A_log, "A_log");
    KDA_OPTIONAL_PTR(S0, "S0");
    KDA_OPTIONAL_PTR(S_out, "S_out");
    KDA_OPTIONAL_PTR(cu_seqlens, "cu_seqlens");
    return KDA_OK;
}
}  // namespace kda

extern "C" {

kda_status_t kda_fwd_chunked(const void* q, const void* k, const void* v, const void* beta,
                             const void* z, const float* A_log, float g_min, const float* S0,
                             float* S_out, const int32_t* cu_seqlens, int N, int64_t T_total,
                             int H, int dk, int dv, kda_dtype_t io_dt, void* o, void* workspace,
                             size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    if (kda_status_t s = kda::check_fwd_args(q, k, v, beta, z, A_log, g_min, S0, S_out,
                                             cu_seqlens, N, T_total, H, dk, dv, io_dt, o))
        return s;
    if (N == 0) return KDA_OK;
    const size_t need = kda_fwd_workspace_size(T_total, N, H, dk, dv, io_dt);
    if (need > 0) {
        KDA_REQUIRE_PTR(workspace, "workspace");
        KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed",
                    ws_bytes, need);
    }

    kda::FwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.z = z;
    a.A_log = A_log; a.g_min = g_min; a.S0 = S0; a.S_out = S_out;
    a.cu_seqlens = cu_seqlens; a.N = N; a.T_total = T_total; a.H = H; a.dk = dk; a.dv = dv;
    a.io_bf16 = (io_dt == KDA_BF16); a.o = o; a.workspace = workspace; a.ws_bytes = ws_bytes;
    a.dev_err = device_error_ptr();
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e =
        use_tc_path(dk, dv, io_dt) ? kda::launch_fwd_tc(a) : kda::launch_fwd_generic(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_fwd_chunked launch");
    return KDA_OK;
}

kda_status_t kda_fwd_chunked_softplus(const void* q, const void* k, const void* v,
                                      const void* beta, const void* z, const float* A_log,
                                      const float* S0, float* S_out, const int32_t* cu_seqlens,
                                      int N, int64_t T_total, int H, int dk, int dv,
                                      kda_dtype_t io_dt, void* o, void* workspace,
                                      size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(N >= 0, "N=%d must be >= 0", N);
    KDA_REQUIRE(H > 0, "H=%d must be positive", H);
    KDA_REQUIRE(T_total >= 0, "T_total=%lld must be >= 0", (long long)T_total);
    if (kda_status_t s = check_dims(dk, dv)) return s;
    if (cu_seqlens == nullptr) {
        KDA_REQUIRE(N > 0 || T_total == 0, "N=0 requires T_total=0");
        KDA_REQUIRE(N == 0 || T_total % N == 0,
                    "without cu_seqlens T_total=%lld must be a multiple of N=%d",
                    (long long)T_total, N);
    }
    KDA_REQUIRE((int64_t)N * H * 4 < (int64_t)1 << 31, "N*H=%lld is too large",
                (long long)N * H);
    if (N == 0) return KDA_OK;
    if (T_total > 0) {
        KDA_REQUIRE_PTR(q, "q");
        KDA_REQUIRE_PTR(k, "k");
        KDA_REQUIRE_PTR(v, "v");
        KDA_REQUIRE_PTR(z, "z");
        KDA_REQUIRE_PTR(o, "o");
        KDA_REQUIRE(beta != nullptr, "beta is NULL");
    }
    KDA_REQUIRE_PTR(A_log, "A_log");
    KDA_OPTIONAL_PTR(S0, "S0");
    KDA_OPTIONAL_PTR(S_out, "S_out");
    KDA_OPTIONAL_PTR(cu_seqlens, "cu_seqlens");
    const size_t need = kda_fwd_workspace_size(T_total, N, H, dk, dv, io_dt);
    if (need > 0) {
        KDA_REQUIRE_PTR(workspace, "workspace");
        KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed",
                    ws_bytes, need);
    }
    kda::FwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.z = z;
    a.A_log = A_log; a.g_min = -1.f; a.S0 = S0; a.S_out = S_out;
    a.cu_seqlens = cu_seqlens; a.N = N; a.T_total = T_total; a.H = H; a.dk = dk; a.dv = dv;
    a.io_bf16 = (io_dt == KDA_BF16); a.gate_kind = 1; a.o = o;
    a.workspace = workspace; a.ws_bytes = ws_bytes;
    a.dev_err = device_error_ptr();
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    // bf16: the mixed path (tensor cores off the diagonal sub-tiles); fp32: the explicit
    // per-pair path
    cudaError_t e =
        use_tc_path(dk, dv, io_dt) ? kda::launch_fwd_tc(a) : kda::launch_fwd_generic(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_fwd_chunked_softplus launch");
    return KDA_OK;
}

size_t kda_bwd_workspace_size(int64_t T_total, int N, int H, int dk, int dv) {
    if (T_total < 0 || N <= 0 || H <= 0 || check_dims(dk, dv) != KDA_OK) return 0;
    return kda::bwd_workspace_size_public(T_total, N, H, dk, dv);
}

kda_status_t kda_bwd(const void* q, const void* k, const void* v, const void* beta,
                     const void* z, const float* A_log, float g_min, const float* S0,
                     const int32_t* cu_seqlens, int N, int64_t T_total, int H, int dk, int dv,
                     kda_dtype_t io_dt, const void* dout, const float* dS_out, void* dq,
                     void* dk_out, void* dv_out, void* dbeta, void* dz, float* dA_log,
                     float* dS0, void* workspace, size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(N > 0, "N=%d must be positive", N);
    KDA_REQUIRE(H > 0, "H=%d must be positive", H);
    KDA_REQUIRE(T_total >= 0, "T_total=%lld must be >= 0", (long long)T_total);
    if (kda_status_t s = check_dims(dk, dv)) return s;
    if (kda_status_t s = check_gmin(g_min)) return s;
    if (cu_seqlens == nullptr)
        KDA_REQUIRE(T_total % N == 0, "without cu_seqlens T_total=%lld must be a multiple of N=%d",
                    (long long)T_total, N);
    KDA_REQUIRE((int64_t)N * H < (int64_t)1 << 31, "N*H=%lld is too large", (long long)N * H);
    if (T_total > 0) {
        KDA_REQUIRE_PTR(q, "q");
        KDA_REQUIRE_PTR(k, "k");
        KDA_REQUIRE_PTR(v, "v");
        KDA_REQUIRE_PTR(z, "z");
        KDA_REQUIRE_PTR(dout, "dout");
        KDA_REQUIRE_PTR(dq, "dq");
        KDA_REQUIRE_PTR(dk_out, "dk");
        KDA_REQUIRE_PTR(dv_out, "dv");
        KDA_REQUIRE_PTR(dz, "dz");
        KDA_REQUIRE(beta != nullptr, "beta is NULL");
        KDA_REQUIRE(dbeta != nullptr, "dbeta is NULL");
    }
    KDA_REQUIRE_PTR(A_log, "A_log");
    KDA_REQUIRE_PTR(dA_log, "dA_log");
    KDA_OPTIONAL_PTR(S0, "S0");
    KDA_OPTIONAL_PTR(dS_out, "dS_out");
    KDA_OPTIONAL_PTR(dS0, "dS0");
    KDA_OPTIONAL_PTR(cu_seqlens, "cu_seqlens");
    const size_t need = kda::bwd_workspace_size_public(T_total, N, H, dk, dv);
    KDA_REQUIRE_PTR(workspace, "workspace");
    KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed",
                ws_bytes, need);
    kda::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.z = z; a.dout = dout;
    a.A_log = A_log; a.g_min = g_min; a.S0 = S0; a.dS_out = dS_out; a.cu_seqlens = cu_seqlens;
    a.N = N; a.T_total = T_total; a.H = H; a.dk = dk; a.dv = dv; a.io_bf16 = io_dt == KDA_BF16;
    a.dq = dq; a.dk_ = dk_out; a.dv_ = dv_out; a.dbeta = dbeta; a.dz = dz; a.dA_log = dA_log;
    a.dS0 = dS0; a.workspace = workspace; a.dev_err = device_error_ptr();
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_bwd(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_bwd launch");
    return KDA_OK;
}

kda_status_t kda_decode_step(const void* q, const void* k, const void* v, const void* beta,
                             const void* z, const float* A_log, float g_min, float* S, int N,
                             int H, int dk, int dv, kda_dtype_t io_dt, void* o,
                             kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(N >= 0, "N=%d must be >= 0", N);
    KDA_REQUIRE(H > 0, "H=%d must be positive", H);
    if (kda_status_t s = check_dims(dk, dv)) return s;
    if (kda_status_t s = check_gmin(g_min)) return s;
    KDA_REQUIRE((int64_t)N * H < (int64_t)1 << 31, "N*H=%lld is too large", (long long)N * H);
    if (N == 0) return KDA_OK;
    KDA_REQUIRE_PTR(q, "q");
    KDA_REQUIRE_PTR(k, "k");
    KDA_REQUIRE_PTR(v, "v");
    KDA_REQUIRE_PTR(z, "z");
    KDA_REQUIRE_PTR(o, "o");
    KDA_REQUIRE_PTR(S, "S");
    KDA_REQUIRE_PTR(A_log, "A_log");
    KDA_REQUIRE(beta != nullptr, "beta is NULL");
    cudaError_t e = kda::launch_decode(q, k, v, beta, z, A_log, g_min, S, N, H, dk, dv,
                                       io_dt == KDA_BF16, o,
                                       reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_decode_step launch");
    return KDA_OK;
}

kda_status_t kda_output_norm_gate(const void* o, const void* gate, const float* norm_w,
                                  float eps, void* y, int64_t n_tokens, int H, int dv,
                                  kda_dtype_t io_dt, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(n_tokens >= 0, "n_tokens=%lld must be >= 0", (long long)n_tokens);
    KDA_REQUIRE(H > 0, "H=%d must be positive", H);
    KDA_REQUIRE(dv > 0, "dv=%d must be positive", dv);
    if (dv != 64 && dv != 128) return fail(KDA_ERR_UNSUPPORTED, "dv=%d: only 64 and 128 are supported", dv);
    KDA_REQUIRE(eps >= 0.f && std::isfinite(eps), "eps=%g must be finite and >= 0", (double)eps);
    if (n_tokens == 0) return KDA_OK;
    KDA_REQUIRE_PTR(o, "o");
    KDA_REQUIRE_PTR(gate, "gate");
    KDA_REQUIRE_PTR(y, "y");
    KDA_OPTIONAL_PTR(norm_w, "norm_w");
    cudaError_t e = kda::launch_output_gate(o, gate, norm_w, eps, y, n_tokens * H, dv,
                                            io_dt == KDA_BF16,
                                            reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_output_norm_gate launch");
    return KDA_OK;
}

kda_status_t kda_decode_step_gated(const void* q, const void* k, const void* v,
                                   const void* beta, const void* z, const float* A_log,
                                   float g_min, float* S, const void* gate, const float* norm_w,
                                   float eps, int N, int H, int dk, int dv, kda_dtype_t io_dt,
                                   void* y, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(N >= 0, "N=%d must be >= 0", N);
    KDA_REQUIRE(H > 0, "H=%d must be positive", H);
    if (kda_status_t s = check_dims(dk, dv)) return s;
    if (kda_status_t s = check_gmin(g_min)) return s;
    KDA_REQUIRE(eps >= 0.f && std::isfinite(eps), "eps=%g must be finite and >= 0", (double)eps);
    KDA_REQUIRE((int64_t)N * H < (int64_t)1 << 31, "N*H=%lld is too large", (long long)N * H);
    if (N == 0) return KDA_OK;
    KDA_REQUIRE_PTR(q, "q");
    KDA_REQUIRE_PTR(k, "k");
    KDA_REQUIRE_PTR(v, "v");
    KDA_REQUIRE_PTR(z, "z");
    KDA_REQUIRE_PTR(gate, "gate");
    KDA_REQUIRE_PTR(y, "y");
    KDA_REQUIRE_PTR(S, "S");
    KDA_REQUIRE_PTR(A_log, "A_log");
    KDA_OPTIONAL_PTR(norm_w, "norm_w");
    KDA_REQUIRE(beta != nullptr, "beta is NULL");
    cudaError_t e = kda::launch_decode_gated(q, k, v, beta, z, A_log, g_min, S, N, H, dk, dv,
                                             io_dt == KDA_BF16, gate, norm_w, eps, y,
                                             reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_decode_step_gated launch");
    return KDA_OK;
}

// Checks shared by the entry points of the per-head-decay linear attention.  A token stride is
// at least a token's heads and a whole number of 16-byte pieces.
static kda_status_t check_linear(int H, int dk, int dv, kda_dtype_t io_dt, int64_t q_ld,
                                 int64_t k_ld, int64_t v_ld) {
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(H > 0 && H <= 65535, "H=%d must be in [1, 65535]", H);
    if (kda_status_t s = check_dims(dk, dv)) return s;
    const int per16 = io_dt == KDA_BF16 ? 8 : 4;
    KDA_REQUIRE(q_ld >= (int64_t)H * dk && q_ld % per16 == 0,
                "q_ld=%lld must be a multiple of %d and at least H dk", (long long)q_ld, per16);
    KDA_REQUIRE(k_ld >= (int64_t)H * dk && k_ld % per16 == 0,
                "k_ld=%lld must be a multiple of %d and at least H dk", (long long)k_ld, per16);
    KDA_REQUIRE(v_ld >= (int64_t)H * dv && v_ld % per16 == 0,
                "v_ld=%lld must be a multiple of %d and at least H dv", (long long)v_ld, per16);
    return KDA_OK;
}

static kda_status_t check_sequences(int64_t T_total, int N, const int32_t* cu_seqlens) {
    KDA_REQUIRE(N >= 0, "N=%d must be >= 0", N);
    KDA_REQUIRE(T_total >= 0 && T_total < (int64_t)1 << 31, "T_total=%lld must be in [0, 2^31)",
                (long long)T_total);
    KDA_REQUIRE(N > 0 || T_total == 0, "N=0 requires T_total=0");
    KDA_REQUIRE(cu_seqlens != nullptr || N == 0 || T_total % N == 0,
                "without cu_seqlens T_total=%lld must be a multiple of N=%d", (long long)T_total,
                N);
    KDA_OPTIONAL_PTR(cu_seqlens, "cu_seqlens");
    return KDA_OK;
}
static kda_status_t check_packed(int64_t T_total, int N, int H, const int32_t* cu_seqlens) {
    if (kda_status_t s = check_sequences(T_total, N, cu_seqlens)) return s;
    KDA_REQUIRE((int64_t)N * H * 4 < (int64_t)1 << 31, "N*H=%lld is too large",
                (long long)N * H);
    return KDA_OK;
}

size_t kda_linear_fwd_workspace_size(int64_t T_total, int N, int H, int dk, int dv,
                                     kda_dtype_t io_dt) {
    if (T_total < 0 || N <= 0 || H <= 0 || check_dims(dk, dv) != KDA_OK) return 0;
    return kda::linear_fwd_workspace_size(T_total, N, H, dk, dv, io_dt == KDA_BF16);
}

size_t kda_linear_bwd_workspace_size(int64_t T_total, int N, int H, int dk, int dv,
                                     kda_dtype_t io_dt) {
    if (T_total < 0 || N <= 0 || H <= 0 || check_dims(dk, dv) != KDA_OK) return 0;
    return kda::linear_bwd_workspace_size(T_total, N, H, dk, dv, io_dt == KDA_BF16);
}

kda_status_t kda_linear_fwd_chunked(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                    const void* v, int64_t v_ld, const float* g, int g_per_token,
                                    const float* S0, float* S_out, const int32_t* cu_seqlens,
                                    int N, int64_t T_total, int H, int dk, int dv,
                                    kda_dtype_t io_dt, void* o, void* workspace, size_t ws_bytes,
                                    kda_stream_t stream) {
    t_last_error.clear();
    if (kda_status_t s = check_linear(H, dk, dv, io_dt, q_ld, k_ld, v_ld)) return s;
    if (kda_status_t s = check_packed(T_total, N, H, cu_seqlens)) return s;
    if (N == 0) return KDA_OK;
    if (T_total > 0) {
        KDA_REQUIRE_PTR(q, "q");
        KDA_REQUIRE_PTR(k, "k");
        KDA_REQUIRE_PTR(v, "v");
        KDA_REQUIRE_WORDS(g, "g");
        KDA_REQUIRE_PTR(o, "o");
    }
    KDA_OPTIONAL_PTR(S0, "S0");
    KDA_OPTIONAL_PTR(S_out, "S_out");
    const size_t need = kda_linear_fwd_workspace_size(T_total, N, H, dk, dv, io_dt);
    if (need > 0) {
        KDA_REQUIRE_PTR(workspace, "workspace");
        KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed",
                    ws_bytes, need);
    }
    kda::LinearArgs a{};
    a.q = q; a.q_ld = q_ld; a.k = k; a.k_ld = k_ld; a.v = v; a.v_ld = v_ld;
    a.g = g; a.g_per_token = g_per_token != 0; a.S0 = S0; a.S_out = S_out;
    a.cu_seqlens = cu_seqlens; a.N = N; a.T_total = T_total; a.H = H; a.dk = dk; a.dv = dv;
    a.io_bf16 = io_dt == KDA_BF16; a.o = o; a.workspace = workspace;
    a.dev_err = device_error_ptr();
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_linear_fwd(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_linear_fwd_chunked launch");
    return KDA_OK;
}

kda_status_t kda_linear_bwd(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                            const void* v, int64_t v_ld, const float* g, int g_per_token,
                            const float* S0, const int32_t* cu_seqlens, int N, int64_t T_total,
                            int H, int dk, int dv, kda_dtype_t io_dt, const void* dout,
                            int64_t dout_ld, const float* dS_out, void* dq, void* dk_out,
                            void* dv_out, float* dg, float* dS0, void* workspace,
                            size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    if (kda_status_t s = check_linear(H, dk, dv, io_dt, q_ld, k_ld, v_ld)) return s;
    if (kda_status_t s = check_packed(T_total, N, H, cu_seqlens)) return s;
    const int per16 = io_dt == KDA_BF16 ? 8 : 4;
    KDA_REQUIRE(dout_ld >= (int64_t)H * dv && dout_ld % per16 == 0,
                "dout_ld=%lld must be a multiple of %d and at least H dv", (long long)dout_ld,
                per16);
    if (dg) KDA_REQUIRE_WORDS(dg, "dg");
    if (N == 0) {  // (a decay that all tokens share has a gradient all the same)
        if (dg == nullptr || g_per_token) return KDA_OK;
        cudaError_t e =
            cudaMemsetAsync(dg, 0, H * sizeof(float), reinterpret_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "kda_linear_bwd");
    }
    if (T_total > 0) {
        KDA_REQUIRE_PTR(q, "q");
        KDA_REQUIRE_PTR(k, "k");
        KDA_REQUIRE_PTR(v, "v");
        KDA_REQUIRE_WORDS(g, "g");
        KDA_REQUIRE_PTR(dout, "dout");
        KDA_REQUIRE_PTR(dq, "dq");
        KDA_REQUIRE_PTR(dk_out, "dk");
        KDA_REQUIRE_PTR(dv_out, "dv");
    }
    KDA_OPTIONAL_PTR(S0, "S0");
    KDA_OPTIONAL_PTR(dS_out, "dS_out");
    KDA_OPTIONAL_PTR(dS0, "dS0");
    const size_t need = kda_linear_bwd_workspace_size(T_total, N, H, dk, dv, io_dt);
    if (need > 0) {
        KDA_REQUIRE_PTR(workspace, "workspace");
        KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed",
                    ws_bytes, need);
    }
    kda::LinearArgs a{};
    a.q = q; a.q_ld = q_ld; a.k = k; a.k_ld = k_ld; a.v = v; a.v_ld = v_ld;
    a.g = g; a.g_per_token = g_per_token != 0; a.S0 = S0;
    a.cu_seqlens = cu_seqlens; a.N = N; a.T_total = T_total; a.H = H; a.dk = dk; a.dv = dv;
    a.io_bf16 = io_dt == KDA_BF16; a.dout = dout; a.dout_ld = dout_ld; a.dS_out = dS_out;
    a.dq = dq; a.dk_ = dk_out; a.dv_ = dv_out; a.dg = dg; a.dS0 = dS0;
    a.workspace = workspace; a.dev_err = device_error_ptr();
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_linear_bwd(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_linear_bwd launch");
    return KDA_OK;
}

kda_status_t kda_linear_decode_step(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                    const void* v, int64_t v_ld, const float* g, int g_per_token,
                                    float* S, const int32_t* slots, int n_slots, int N, int H,
                                    int dk, int dv, kda_dtype_t io_dt, void* o,
                                    kda_stream_t stream) {
    t_last_error.clear();
    if (kda_status_t s = check_linear(H, dk, dv, io_dt, q_ld, k_ld, v_ld)) return s;
    KDA_REQUIRE(N >= 0, "N=%d must be >= 0", N);
    KDA_REQUIRE((int64_t)N * H < (int64_t)1 << 31, "N*H=%lld is too large", (long long)N * H);
    KDA_REQUIRE(n_slots >= 0, "n_slots=%d must be >= 0", n_slots);
    KDA_REQUIRE(slots != nullptr || n_slots >= N, "n_slots=%d must be at least N=%d without slots",
                n_slots, N);
    if (N == 0) return KDA_OK;
    KDA_REQUIRE_PTR(q, "q");
    KDA_REQUIRE_PTR(k, "k");
    KDA_REQUIRE_PTR(v, "v");
    KDA_REQUIRE_WORDS(g, "g");
    KDA_REQUIRE_PTR(S, "S");
    KDA_REQUIRE_PTR(o, "o");
    if (slots) KDA_REQUIRE_WORDS(slots, "slots");
    unsigned* err = device_error_ptr();
    if (err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_linear_decode(q, q_ld, k, k_ld, v, v_ld, g, g_per_token != 0, S,
                                              slots, n_slots, N, H, dk, dv, io_dt == KDA_BF16, o,
                                              err, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_linear_decode_step launch");
    return KDA_OK;
}

static kda_status_t check_qk_norm(const kda::QkNormArgs& a, kda_dtype_t io_dt, bool bwd) {
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(a.T >= 0 && a.T < (int64_t)1 << 31, "T=%lld must be in [0, 2^31)", (long long)a.T);
    KDA_REQUIRE(a.Hq > 0 && a.Hq <= 65535, "Hq=%d must be in [1, 65535]", a.Hq);
    KDA_REQUIRE(a.Hk >= 0 && a.Hk <= 65535, "Hk=%d must be in [0, 65535]", a.Hk);
    if (a.d != 64 && a.d != 128)
        return fail(KDA_ERR_UNSUPPORTED, "d=%d: only 64 and 128 are supported", a.d);
    KDA_REQUIRE(a.rot_dim >= 0 && a.rot_dim <= a.d, "rot_dim=%d must be in [0, %d]", a.rot_dim,
                a.d);
    if (a.rot_dim % 16 != 0)
        return fail(KDA_ERR_UNSUPPORTED, "rot_dim=%d: only multiples of 16 are supported",
                    a.rot_dim);
    KDA_REQUIRE(a.eps >= 0.f && std::isfinite(a.eps), "eps=%g must be finite and >= 0",
                (double)a.eps);
    const int per16 = io_dt == KDA_BF16 ? 8 : 4;
    KDA_REQUIRE(a.q_ld >= (int64_t)a.Hq * a.d && a.q_ld % per16 == 0,
                "q_ld=%lld must be a multiple of %d and at least Hq d", (long long)a.q_ld, per16);
    KDA_REQUIRE(a.Hk == 0 || (a.k_ld >= (int64_t)a.Hk * a.d && a.k_ld % per16 == 0),
                "k_ld=%lld must be a multiple of %d and at least Hk d", (long long)a.k_ld, per16);
    KDA_OPTIONAL_PTR(a.wq, "wq");
    KDA_OPTIONAL_PTR(a.wk, "wk");
    if (a.rot_dim > 0) {
        KDA_REQUIRE_PTR(a.cos_sin, "cos_sin");
        if (a.positions) KDA_REQUIRE_WORDS(a.positions, "positions");
        KDA_REQUIRE(a.n_pos >= 0, "n_pos=%lld must be >= 0", (long long)a.n_pos);
        KDA_REQUIRE(a.positions != nullptr || a.n_pos >= a.T,
                    "n_pos=%lld must be at least T=%lld without positions", (long long)a.n_pos,
                    (long long)a.T);
    }
    if (a.T > 0) {
        KDA_REQUIRE_PTR(a.q, "q");
        if (bwd) KDA_REQUIRE_PTR(a.dyq, "dyq");
        KDA_REQUIRE_PTR(a.q_out, bwd ? "dq" : "q_out");
        if (a.Hk > 0) {
            KDA_REQUIRE_PTR(a.k, "k");
            if (bwd) KDA_REQUIRE_PTR(a.dyk, "dyk");
            KDA_REQUIRE_PTR(a.k_out, bwd ? "dk" : "k_out");
        }
    }
    return KDA_OK;
}

kda_status_t kda_qk_norm_rope(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                              const float* wq, const float* wk, float eps, const float* cos_sin,
                              int64_t n_pos, const int32_t* positions, int rot_dim,
                              int interleaved, void* q_out, void* k_out, int64_t T, int Hq,
                              int Hk, int d, kda_dtype_t io_dt, kda_stream_t stream) {
    t_last_error.clear();
    kda::QkNormArgs a{};
    a.q = q; a.q_ld = q_ld; a.k = k; a.k_ld = k_ld; a.wq = wq; a.wk = wk; a.eps = eps;
    a.cos_sin = cos_sin; a.n_pos = n_pos; a.positions = positions; a.rot_dim = rot_dim;
    a.interleaved = interleaved != 0; a.q_out = q_out; a.k_out = k_out; a.T = T; a.Hq = Hq;
    a.Hk = Hk; a.d = d; a.io_bf16 = io_dt == KDA_BF16;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (kda_status_t s = check_qk_norm(a, io_dt, false)) return s;
    KDA_REQUIRE(q_out != q || q_ld == (int64_t)Hq * d, "q_out may be q only where q is contiguous");
    KDA_REQUIRE(Hk == 0 || k_out != k || k_ld == (int64_t)Hk * d,
                "k_out may be k only where k is contiguous");
    if (T == 0) return KDA_OK;
    a.dev_err = device_error_ptr();
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_qk_norm(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_qk_norm_rope launch");
    return KDA_OK;
}

size_t kda_qk_norm_rope_bwd_workspace_size(int d) {
    return d == 64 || d == 128 ? kda::qk_norm_bwd_workspace_size(d) : 0;
}

kda_status_t kda_qk_norm_rope_bwd(const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                  const void* dyq, const void* dyk, const float* wq,
                                  const float* wk, float eps, const float* cos_sin,
                                  int64_t n_pos, const int32_t* positions, int rot_dim,
                                  int interleaved, void* dq, void* dk_out, float* dwq,
                                  float* dwk, int64_t T, int Hq, int Hk, int d,
                                  kda_dtype_t io_dt, void* workspace, size_t ws_bytes,
                                  kda_stream_t stream) {
    t_last_error.clear();
    kda::QkNormArgs a{};
    a.q = q; a.q_ld = q_ld; a.k = k; a.k_ld = k_ld; a.dyq = dyq; a.dyk = dyk; a.wq = wq;
    a.wk = wk; a.eps = eps; a.cos_sin = cos_sin; a.n_pos = n_pos; a.positions = positions;
    a.rot_dim = rot_dim; a.interleaved = interleaved != 0; a.q_out = dq; a.k_out = dk_out;
    a.dwq = dwq; a.dwk = dwk; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d;
    a.io_bf16 = io_dt == KDA_BF16; a.workspace = workspace;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (kda_status_t s = check_qk_norm(a, io_dt, true)) return s;
    KDA_OPTIONAL_PTR(dwq, "dwq");
    KDA_OPTIONAL_PTR(dwk, "dwk");
    if (dwq || dwk) {
        const size_t need = kda::qk_norm_bwd_workspace_size(d);
        KDA_REQUIRE_PTR(workspace, "workspace");
        KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed",
                    ws_bytes, need);
    }
    a.dev_err = device_error_ptr();
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_qk_norm_bwd(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_qk_norm_rope_bwd launch");
    return KDA_OK;
}

// ------------------------------------- recurrence of single channels --

static kda_status_t check_width(int D) {
    KDA_REQUIRE(D > 0, "D=%d must be positive", D);
    if (D % 8 != 0) return fail(KDA_ERR_UNSUPPORTED, "D=%d: only multiples of 8 are supported", D);
    return KDA_OK;
}

static kda_status_t check_ld(int64_t ld, int D, int per16, const char* name) {
    KDA_REQUIRE(ld >= D && ld % per16 == 0, "%s=%lld must be a multiple of %d and at least D", name,
                (long long)ld, per16);
    return KDA_OK;
}

// (rows of states are addressed in 64 bits)
static kda_status_t check_states(int N, int D) {
    KDA_REQUIRE((int64_t)N * D < (int64_t)1 << 36, "N*D=%lld is too large", (long long)N * D);
    return KDA_OK;
}

// What the forward and both backward entries share, the workspace excepted.
static kda_status_t check_recurrence(const kda::RecurrenceArgs& a, kda_dtype_t io_dt) {
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    if (kda_status_t s = check_width(a.D)) return s;
    if (kda_status_t s = check_gmin(a.g_min)) return s;
    if (kda_status_t s = check_sequences(a.T_total, a.N, a.cu_seqlens)) return s;
    if (kda_status_t s = check_states(a.N, a.D)) return s;
    // (tokens are counted in 32 bits, those of tiles behind the last one too)
    KDA_REQUIRE(a.T_total < ((int64_t)1 << 31) - 2048, "T_total=%lld must be below 2^31 - 2048",
                (long long)a.T_total);
    const int per16 = io_dt == KDA_BF16 ? 8 : 4;
    if (!a.packed) {
        if (kda_status_t s = check_ld(a.x_ld, a.D, per16, "x_ld")) return s;
        if (kda_status_t s = check_ld(a.z_ld, a.D, per16, "z_ld")) return s;
        if (kda_status_t s = check_ld(a.i_ld, a.D, per16, "i_ld")) return s;
    }
    if (a.T_total > 0) {
        KDA_REQUIRE_PTR(a.x, a.packed ? "x_codes" : "x");
        KDA_REQUIRE_PTR(a.z, a.packed ? "z_codes" : "z");
        KDA_REQUIRE_PTR(a.i, a.packed ? "i_codes" : "i");
        if (a.packed) {
            KDA_REQUIRE(a.x_exps != nullptr, "x_exps is NULL");
            KDA_REQUIRE(a.z_exps != nullptr, "z_exps is NULL");
            KDA_REQUIRE(a.i_exps != nullptr, "i_exps is NULL");
        }
        KDA_REQUIRE_PTR(a.A_log, "A_log");
    }
    KDA_OPTIONAL_PTR(a.h0, "h0");
    KDA_OPTIONAL_PTR(a.edges, "edges");
    return KDA_OK;
}

static kda_status_t check_workspace(const void* workspace, size_t ws_bytes, size_t need) {
    if (need == 0) return KDA_OK;
    KDA_REQUIRE_PTR(workspace, "workspace");
    KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes,
                need);
    return KDA_OK;
}

size_t kda_recurrence_fwd_workspace_size(int64_t T_total, int N, int D) {
    if (T_total < 0 || N <= 0 || D <= 0 || D % 8 != 0) return 0;
    return kda::recurrence_fwd_workspace_size(T_total, N, D);
}

size_t kda_recurrence_bwd_workspace_size(int64_t T_total, int N, int D) {
    if (T_total < 0 || N <= 0 || D <= 0 || D % 8 != 0) return 0;
    return kda::recurrence_bwd_workspace_size(T_total, N, D);
}

kda_status_t kda_recurrence_fwd(const void* x, int64_t x_ld, const void* z, int64_t z_ld,
                                const void* i, int64_t i_ld, const float* A_log, float g_min,
                                const float* h0, float* h_out, const int32_t* cu_seqlens, int N,
                                int64_t T_total, int D, kda_dtype_t io_dt, void* y, float* edges,
                                void* workspace, size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    kda::RecurrenceArgs a{};
    a.x = x; a.x_ld = x_ld; a.z = z; a.z_ld = z_ld; a.i = i; a.i_ld = i_ld; a.A_log = A_log;
    a.g_min = g_min; a.h0 = h0; a.h_out = h_out; a.cu_seqlens = cu_seqlens; a.N = N;
    a.T_total = T_total; a.D = D; a.io_bf16 = io_dt == KDA_BF16; a.y = y; a.edges = edges;
    a.workspace = workspace; a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (kda_status_t s = check_recurrence(a, io_dt)) return s;
    if (N == 0) return KDA_OK;
    if (T_total > 0) KDA_REQUIRE_PTR(y, "y");
    KDA_OPTIONAL_PTR(h_out, "h_out");
    if (kda_status_t s = check_workspace(workspace, ws_bytes,
                                         kda_recurrence_fwd_workspace_size(T_total, N, D)))
        return s;
    a.dev_err = device_error_ptr();
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_recurrence_fwd(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_recurrence_fwd launch");
    return KDA_OK;
}

static kda_status_t recurrence_bwd(kda::RecurrenceArgs& a, kda_dtype_t io_dt, size_t ws_bytes,
                                   const char* where) {
    if (kda_status_t s = check_recurrence(a, io_dt)) return s;
    if (kda_status_t s = check_ld(a.dy_ld, a.D, io_dt == KDA_BF16 ? 8 : 4, "dy_ld")) return s;
    if (a.T_total > 0) {
        KDA_REQUIRE_PTR(a.dy, "dy");
        KDA_REQUIRE_PTR(a.dx, "dx");
        KDA_REQUIRE_PTR(a.dz, "dz");
        KDA_REQUIRE_PTR(a.di, "di");
    }
    KDA_OPTIONAL_PTR(a.dh_out, "dh_out");
    KDA_OPTIONAL_PTR(a.dA_log, "dA_log");
    KDA_OPTIONAL_PTR(a.dh0, "dh0");
    if (a.N == 0) {  // (A_log, which all tokens share, has a gradient all the same)
        if (a.dA_log == nullptr) return KDA_OK;
        cudaError_t e = cudaMemsetAsync(a.dA_log, 0, a.D * sizeof(float), a.stream);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, where);
    }
    if (kda_status_t s = check_workspace(
            a.workspace, ws_bytes, kda_recurrence_bwd_workspace_size(a.T_total, a.N, a.D)))
        return s;
    a.dev_err = device_error_ptr();
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_recurrence_bwd(a);
    if (e != cudaSuccess) return cuda_fail(e, where);
    return KDA_OK;
}

kda_status_t kda_recurrence_bwd(const void* x, int64_t x_ld, const void* z, int64_t z_ld,
                                const void* i, int64_t i_ld, const float* A_log, float g_min,
                                const float* h0, const int32_t* cu_seqlens, int N,
                                int64_t T_total, int D, kda_dtype_t io_dt, const void* dy,
                                int64_t dy_ld, const float* dh_out, const float* edges, void* dx,
                                void* dz, void* di, float* dA_log, float* dh0, void* workspace,
                                size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    kda::RecurrenceArgs a{};
    a.x = x; a.x_ld = x_ld; a.z = z; a.z_ld = z_ld; a.i = i; a.i_ld = i_ld; a.A_log = A_log;
    a.g_min = g_min; a.h0 = h0; a.cu_seqlens = cu_seqlens; a.N = N; a.T_total = T_total; a.D = D;
    a.io_bf16 = io_dt == KDA_BF16; a.dy = dy; a.dy_ld = dy_ld; a.dh_out = dh_out;
    a.edges = const_cast<float*>(edges); a.dx = dx; a.dz = dz; a.di = di; a.dA_log = dA_log;
    a.dh0 = dh0; a.workspace = workspace; a.stream = reinterpret_cast<cudaStream_t>(stream);
    return recurrence_bwd(a, io_dt, ws_bytes, "kda_recurrence_bwd launch");
}

kda_status_t kda_recurrence_bwd_packed(const int8_t* x_codes, const int8_t* x_exps,
                                       const int8_t* z_codes, const int8_t* z_exps,
                                       const int8_t* i_codes, const int8_t* i_exps,
                                       const float* A_log, float g_min, const float* h0,
                                       const int32_t* cu_seqlens, int N, int64_t T_total, int D,
                                       kda_dtype_t io_dt, const void* dy, int64_t dy_ld,
                                       const float* dh_out, void* dx, void* dz, void* di,
                                       float* dA_log, float* dh0, void* workspace,
                                       size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    kda::RecurrenceArgs a{};
    a.x = x_codes; a.z = z_codes; a.i = i_codes; a.x_ld = a.z_ld = a.i_ld = D; a.packed = 1;
    a.x_exps = x_exps; a.z_exps = z_exps; a.i_exps = i_exps; a.A_log = A_log; a.g_min = g_min;
    a.h0 = h0; a.cu_seqlens = cu_seqlens; a.N = N; a.T_total = T_total; a.D = D;
    a.io_bf16 = io_dt == KDA_BF16; a.dy = dy; a.dy_ld = dy_ld; a.dh_out = dh_out; a.dx = dx;
    a.dz = dz; a.di = di; a.dA_log = dA_log; a.dh0 = dh0; a.workspace = workspace;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return recurrence_bwd(a, io_dt, ws_bytes, "kda_recurrence_bwd_packed launch");
}

kda_status_t kda_recurrence_step(const void* x, int64_t x_ld, const void* z, int64_t z_ld,
                                 const void* i, int64_t i_ld, const float* A_log, float g_min,
                                 float* h, const int32_t* slots, int n_slots, int N, int D,
                                 kda_dtype_t io_dt, void* y, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    if (kda_status_t s = check_width(D)) return s;
    if (kda_status_t s = check_gmin(g_min)) return s;
    const int per16 = io_dt == KDA_BF16 ? 8 : 4;
    if (kda_status_t s = check_ld(x_ld, D, per16, "x_ld")) return s;
    if (kda_status_t s = check_ld(z_ld, D, per16, "z_ld")) return s;
    if (kda_status_t s = check_ld(i_ld, D, per16, "i_ld")) return s;
    KDA_REQUIRE(N >= 0, "N=%d must be >= 0", N);
    if (kda_status_t s = check_states(N, D)) return s;
    KDA_REQUIRE(n_slots >= 0, "n_slots=%d must be >= 0", n_slots);
    KDA_REQUIRE(slots != nullptr || n_slots >= N, "n_slots=%d must be at least N=%d without slots",
                n_slots, N);
    if (N == 0) return KDA_OK;
    KDA_REQUIRE_PTR(x, "x");
    KDA_REQUIRE_PTR(z, "z");
    KDA_REQUIRE_PTR(i, "i");
    KDA_REQUIRE_PTR(A_log, "A_log");
    KDA_REQUIRE_PTR(h, "h");
    KDA_REQUIRE_PTR(y, "y");
    if (slots) KDA_REQUIRE_WORDS(slots, "slots");
    unsigned* err = device_error_ptr();
    if (err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_recurrence_step(x, x_ld, z, z_ld, i, i_ld, A_log, g_min, h, slots,
                                                n_slots, N, D, io_dt == KDA_BF16, y, err,
                                                reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_recurrence_step launch");
    return KDA_OK;
}

// --------------------------------------------- activations in 8 bits --

static kda_status_t check_checkpoint(int64_t T, int D, kda_dtype_t io_dt) {
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(T >= 0 && T < (int64_t)1 << 31, "T=%lld must be in [0, 2^31)", (long long)T);
    return check_width(D);
}

kda_status_t kda_checkpoint_pack(const void* x, int64_t x_ld, int64_t T, int D,
                                 kda_dtype_t io_dt, int8_t* codes, int8_t* exps,
                                 kda_stream_t stream) {
    t_last_error.clear();
    if (kda_status_t s = check_checkpoint(T, D, io_dt)) return s;
    if (kda_status_t s = check_ld(x_ld, D, io_dt == KDA_BF16 ? 8 : 4, "x_ld")) return s;
    if (T == 0) return KDA_OK;
    KDA_REQUIRE_PTR(x, "x");
    KDA_REQUIRE_PTR(codes, "codes");
    KDA_REQUIRE(exps != nullptr, "exps is NULL");
    cudaError_t e = kda::launch_checkpoint_pack(x, x_ld, T, D, io_dt == KDA_BF16, codes, exps,
                                                reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_checkpoint_pack launch");
    return KDA_OK;
}

kda_status_t kda_checkpoint_unpack(const int8_t* codes, const int8_t* exps, int64_t T, int D,
                                   kda_dtype_t io_dt, void* x, kda_stream_t stream) {
    t_last_error.clear();
    if (kda_status_t s = check_checkpoint(T, D, io_dt)) return s;
    if (T == 0) return KDA_OK;
    KDA_REQUIRE_PTR(codes, "codes");
    KDA_REQUIRE(exps != nullptr, "exps is NULL");
    KDA_REQUIRE_PTR(x, "x");
    cudaError_t e = kda::launch_checkpoint_unpack(codes, exps, T, D, io_dt == KDA_BF16, x,
                                                  reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_checkpoint_unpack launch");
    return KDA_OK;
}

// ---------------------------------------------- norms around a block --

static kda_status_t check_block_norm(const kda::BlockNormArgs& a, kda_dtype_t io_dt,
                                     kda_dtype_t r_dt) {
    KDA_REQUIRE(io_dt == KDA_F32 || io_dt == KDA_BF16, "io_dt=%d is not a kda_dtype_t", (int)io_dt);
    KDA_REQUIRE(r_dt == KDA_F32 || r_dt == io_dt, "r_dt=%d must be io_dt or KDA_F32", (int)r_dt);
    KDA_REQUIRE(a.T >= 0 && a.T < (int64_t)1 << 31, "T=%lld must be in [0, 2^31)", (long long)a.T);
    if (kda_status_t s = check_width(a.D)) return s;
    if (a.D > kda::kMaxBlockNormD)
        return fail(KDA_ERR_UNSUPPORTED, "D=%d: at most %d is supported", a.D, kda::kMaxBlockNormD);
    KDA_REQUIRE(a.eps >= 0.f && std::isfinite(a.eps), "eps=%g must be finite and >= 0",
                (double)a.eps);
    KDA_REQUIRE(a.post_norm || a.w_post == nullptr, "w_post must be NULL without a post-norm");
    KDA_OPTIONAL_PTR(a.gate, "gate");
    KDA_OPTIONAL_PTR(a.scale, "scale");
    KDA_OPTIONAL_PTR(a.w_post, "w_post");
    KDA_OPTIONAL_PTR(a.w_pre, "w_pre");
    return KDA_OK;
}

kda_status_t kda_block_norm(const void* y, const void* gate, const void* r, const float* scale,
                            const float* w_post, const float* w_pre, int post_norm, float eps,
                            void* r_out, void* x_out, int64_t T, int D, kda_dtype_t io_dt,
                            kda_dtype_t r_dt, kda_stream_t stream) {
    t_last_error.clear();
    kda::BlockNormArgs a{};
    a.y = y; a.gate = gate; a.r = r; a.scale = scale; a.w_post = w_post; a.w_pre = w_pre;
    a.post_norm = post_norm != 0; a.eps = eps; a.r_out = r_out; a.x_out = x_out; a.T = T; a.D = D;
    a.io_bf16 = io_dt == KDA_BF16; a.r_bf16 = r_dt == KDA_BF16;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (kda_status_t s = check_block_norm(a, io_dt, r_dt)) return s;
    if (T == 0) return KDA_OK;
    KDA_REQUIRE_PTR(y, "y");
    KDA_REQUIRE_PTR(r, "r");
    KDA_REQUIRE_PTR(r_out, "r_out");
    KDA_REQUIRE_PTR(x_out, "x_out");
    cudaError_t e = kda::launch_block_norm(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_block_norm launch");
    return KDA_OK;
}

size_t kda_block_norm_bwd_workspace_size(int D) {
    if (D <= 0 || D % 8 != 0 || D > kda::kMaxBlockNormD) return 0;
    return kda::block_norm_bwd_workspace_size(D);
}

kda_status_t kda_block_norm_bwd(const void* y, const void* gate, const void* r_out,
                                const void* dx, const void* dr, const float* scale,
                                const float* w_post, const float* w_pre, int post_norm, float eps,
                                void* dr_in, void* dy, void* dgate, float* dscale, float* dw_post,
                                float* dw_pre, int64_t T, int D, kda_dtype_t io_dt,
                                kda_dtype_t r_dt, void* workspace, size_t ws_bytes,
                                kda_stream_t stream) {
    t_last_error.clear();
    kda::BlockNormArgs a{};
    a.y = y; a.gate = gate; a.r = r_out; a.dx = dx; a.dr = dr; a.scale = scale; a.w_post = w_post;
    a.w_pre = w_pre; a.post_norm = post_norm != 0; a.eps = eps; a.dr_in = dr_in; a.dy = dy;
    a.dgate = dgate; a.dscale = dscale; a.dw_post = dw_post; a.dw_pre = dw_pre; a.T = T; a.D = D;
    a.io_bf16 = io_dt == KDA_BF16; a.r_bf16 = r_dt == KDA_BF16; a.workspace = workspace;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (kda_status_t s = check_block_norm(a, io_dt, r_dt)) return s;
    KDA_REQUIRE(post_norm || dw_post == nullptr, "dw_post must be NULL without a post-norm");
    if (T > 0) {
        KDA_REQUIRE_PTR(y, "y");
        KDA_REQUIRE_PTR(r_out, "r_out");
        KDA_REQUIRE_PTR(dx, "dx");
        KDA_OPTIONAL_PTR(dr, "dr");
        KDA_REQUIRE_PTR(dr_in, "dr_in");
        KDA_REQUIRE_PTR(dy, "dy");
        if (gate) KDA_REQUIRE_PTR(dgate, "dgate");
        KDA_REQUIRE(gate || dgate == nullptr, "dgate must be NULL without a gate");
    }
    KDA_OPTIONAL_PTR(dscale, "dscale");
    KDA_OPTIONAL_PTR(dw_post, "dw_post");
    KDA_OPTIONAL_PTR(dw_pre, "dw_pre");
    if (dscale || dw_post || dw_pre)
        if (kda_status_t s =
                check_workspace(workspace, ws_bytes, kda::block_norm_bwd_workspace_size(D)))
            return s;
    a.dev_err = device_error_ptr();
    if (a.dev_err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_block_norm_bwd(a);
    if (e != cudaSuccess) return cuda_fail(e, "kda_block_norm_bwd launch");
    return KDA_OK;
}

size_t kda_quantile_balance_workspace_size(int64_t m, int n) {
    if (m <= 0 || n <= 0) return 0;
    return kda::qb_workspace_size(m, n);
}

kda_status_t kda_quantile_balance(const float* scores, const float* bias, int64_t m, int n,
                                  int k, float* bias_new, float* bhat, float* alpha,
                                  void* workspace, size_t ws_bytes, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(m >= 1 && m < ((int64_t)1 << 31), "m=%lld must be in [1, 2^31)", (long long)m);
    KDA_REQUIRE(n >= 1 && n <= 1024, "n=%d must be in [1, 1024]", n);
    KDA_REQUIRE(k >= 0 && k < n, "k=%d must satisfy 0 <= k < n=%d", k, n);
    KDA_REQUIRE_PTR(scores, "scores");
    KDA_REQUIRE_PTR(bias, "bias");
    KDA_REQUIRE_PTR(bias_new, "bias_new");
    KDA_OPTIONAL_PTR(bhat, "bhat");
    KDA_OPTIONAL_PTR(alpha, "alpha");
    const size_t need = kda::qb_workspace_size(m, n);
    KDA_REQUIRE_PTR(workspace, "workspace");
    KDA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed",
                ws_bytes, need);
    cudaError_t e = kda::launch_quantile_balance(scores, bias, m, n, k, bias_new, bhat, alpha,
                                                 workspace,
                                                 reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_quantile_balance launch");
    return KDA_OK;
}

kda_status_t kda_selftest_timeout(unsigned limit_us, kda_stream_t stream) {
    t_last_error.clear();
    KDA_REQUIRE(limit_us >= 1 && limit_us <= 2000000u, "limit_us=%u must be in [1, 2e6]",
                limit_us);
    unsigned* err = device_error_ptr();
    if (err == nullptr) return fail(KDA_ERR_CUDA, "no CUDA device is usable");
    cudaError_t e = kda::launch_selftest_timeout((uint64_t)limit_us * 1000u, err,
                                                 reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_selftest_timeout launch");
    return KDA_OK;
}

kda_status_t kda_device_status(kda_stream_t stream) {
    t_last_error.clear();
    cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_device_status wait");
    unsigned word = 0u;
    e = cudaMemcpyFromSymbol(&word, g_device_error, sizeof word);
    if (e != cudaSuccess) return cuda_fail(e, "kda_device_status read");
    const unsigned zero = 0u;
    e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
    if (e != cudaSuccess) return cuda_fail(e, "kda_device_status clear");
    if (word & kda::kDevErrTimeout)
        return fail(KDA_ERR_TIMEOUT, "a device-side wait gave up (error word 0x%x)", word);
    if (word & kda::kDevErrBadSeqlens)
        return fail(KDA_ERR_DEVICE, "malformed cu_seqlens met on the device (error word 0x%x)",
                    word);
    if (word & kda::kDevErrBadSlot)
        return fail(KDA_ERR_DEVICE, "a slot outside the pool met on the device (error word 0x%x)",
                    word);
    if (word & kda::kDevErrBadPosition)
        return fail(KDA_ERR_DEVICE,
                    "a position outside the table met on the device (error word 0x%x)", word);
    return KDA_OK;
}

}  // extern "C"
