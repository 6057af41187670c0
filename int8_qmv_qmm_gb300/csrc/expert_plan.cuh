// What the kernels of the experts' products share: the rows of an expert in a
// routing's plan, as far as the plan is what the call says.
#pragma once

#include <stdint.h>

#include "qlin_internal.h"

namespace qlin {

// Bits of the experts' status words.
enum : unsigned {
  kStatusPlan = 1u,  // offsets that are no plan's, or a pair outside n_pairs
  kStatusWait = 2u,  // a wait that gave up
};

struct ExpertRows {
  int first;  // in order
  int n;
  bool bad;   // the offsets are not those of a plan: the expert is left out
};

__device__ __forceinline__ ExpertRows expert_rows(const ExpertArgs& a, int expert) {
  const int first = a.offsets[expert], end = a.offsets[expert + 1];
  ExpertRows r;
  r.bad = first < 0 || end < first || end > a.n_pairs;
  r.first = r.bad ? 0 : first;
  r.n = r.bad ? 0 : end - first;
  return r;
}

// Whether the streaming kernel's tokens fit in shared memory.
bool expert_stream_fits(int64_t K);
qlin_status launch_expert_stream(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st);
cudaError_t expert_stream_take_status(unsigned* flags);
qlin_status launch_expert_tile(const ExpertArgs& a, int bits, qlin_dtype dtype, double rows,
                               unsigned flags, cudaStream_t st);
size_t expert_tile_workspace_size(int64_t n_pairs, int E, int64_t N, int64_t K);
cudaError_t expert_tile_take_status(unsigned* flags);

}  // namespace qlin
