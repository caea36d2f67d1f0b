// linear_tc.h -- host side of linear_tc.cu: bf16 calls of the per-head-decay linear attention on
// the tensor cores (linear_common.cuh has the calls and the segments; segment lengths must be a
// multiple of 128 tokens).
#pragma once

#include "linear_common.cuh"

namespace kda {
namespace lintc {

// What the kernels below need of the decays, once for all calls (`rec` holds record_bytes()), and
// the counters of taken items, zeroed.
constexpr int kCounters = 3;
size_t record_bytes(int64_t T, int N, int H);
cudaError_t launch_decays(const lin::Problem& p, float* rec, unsigned* next, cudaStream_t s);

// Every segment's outputs from its edge state, of calls that all or none want dot products; `next`:
// a zeroed counter.
cudaError_t launch_outputs(const lin::Problem& p, const lin::Calls& calls, int n, int64_t slots,
                           const float* rec, unsigned* next, const char* name, cudaStream_t s);

// kSegments: each segment's own contribution to the state, of the sequences that have several, into
// calls.c[i].seg, and its summed log2 decay into dec[reverse][edge slot][head] (the walk's last
// only for a call with S_out or anchors).  kSingles: the states after the other sequences, from
// .edge, into .S_out and .anchors.  States in memory are [da][db] (tr = 0).
enum { kSegments = 1, kSingles = 2 };
cudaError_t launch_sums(const lin::Problem& p, const lin::Calls& calls, int n, int64_t slots,
                        const float* rec, float* dec, unsigned* next, int sums, const char* name,
                        cudaStream_t s);

}  // namespace lintc
}  // namespace kda
