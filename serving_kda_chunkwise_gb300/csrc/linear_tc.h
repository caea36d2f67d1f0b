// linear_tc.h -- host side of linear_tc.cu: bf16 calls of the per-head-decay linear attention on
// the tensor cores (linear_common.cuh has the calls and the segments; segment lengths must be a
// multiple of 128 tokens).
#pragma once

#include "linear_common.cuh"

namespace kda {
namespace lintc {

// Every segment's outputs (and final states) from its edge state.
cudaError_t launch_outputs(const lin::Problem& p, const lin::Calls& calls, int n, int64_t slots,
                           const char* name, cudaStream_t s);

// Every segment's own contribution to the state into calls.c[i].seg, and its summed log2 decay
// into dec[reverse][slot][head]; states in memory are [da][db] (tr = 0).
cudaError_t launch_sums(const lin::Problem& p, const lin::Calls& calls, int n, int64_t slots,
                        float* dec, const char* name, cudaStream_t s);

}  // namespace lintc
}  // namespace kda
