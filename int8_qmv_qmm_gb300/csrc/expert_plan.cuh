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

// The plan in shared memory, as jobs: an expert's rows in stretches of `tile` tokens.
template <int kMaxExperts>
struct Jobs {
  int first[kMaxExperts + 1];  // the jobs of the experts before each
  int row[kMaxExperts];        // each expert's first place in order
  int count[kMaxExperts];      // and its rows
  int warp_sum[32];
};

// Fills it, by all threads of the CTA, at least kMaxExperts of them (two barriers; a
// thread an expert: a warp that went over them in steps of 32 took 1.5 us for 512).
// Returns whether any expert was left out.
template <int kMaxExperts>
__device__ __forceinline__ bool fill_jobs(const ExpertArgs& a, int tile, Jobs<kMaxExperts>& j) {
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  bool bad = false;
  int jobs = 0;
  if (e < a.E) {
    const ExpertRows r = expert_rows(a, e);
    bad = r.bad;
    j.row[e] = r.first;
    j.count[e] = r.n;
    jobs = (r.n + tile - 1) / tile;
  }
  int upto = jobs;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) j.warp_sum[warp] = upto;
  if (e == 0) j.first[0] = 0;
  __syncthreads();
  if (e < a.E) {
    for (int w = 0; w < warp; ++w) upto += j.warp_sum[w];
    j.first[e + 1] = upto;
  }
  __syncthreads();
  return bad;
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
