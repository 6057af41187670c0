// The experts' products from packed weights (qlin.h has the definition): which kernel
// takes a call.

#include "expert_plan.cuh"
#include "qlin_internal.h"

namespace qlin {

namespace {

// Rows of an expert, were they spread evenly (the routing itself is on the device).
double rows_of(int64_t n_pairs, int E) {
  return double(n_pairs) / double(E < n_pairs ? E : n_pairs);
}

// The streaming kernel takes experts of up to 5 rows, the tensor-core kernel those of more.
// (64 experts, us, streaming and tensor cores: 1024 x 2048 at 8 bits in bf16 with 1, 4, 5
// and 8 rows an expert 20 and 24, 32 and 35, 34 and 35, 45 and 36; 2048 x 2048 at 4 bits in
// f16 with 2, 4 and 5 rows 40 and 52, 48 and 59, 54 and 61; 60 of 1408 x 2501 at 8 bits with
// 10 rows 62 and 49.)
constexpr double kStreamRows = 5.0;

bool streams(int64_t n_pairs, int E, int64_t K) {
  return rows_of(n_pairs, E) <= kStreamRows && expert_stream_fits(K);
}

}  // namespace

size_t expert_linear_workspace_size(int64_t n_pairs, int E, int64_t N, int64_t K) {
  return n_pairs > 0 && !streams(n_pairs, E, K) ? expert_tile_workspace_size(n_pairs, E, N, K) : 0;
}

qlin_status launch_expert_linear(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st) {
  if (streams(a.n_pairs, a.E, a.K)) return launch_expert_stream(a, bits, dtype, flags, st);
  return launch_expert_tile(a, bits, dtype, rows_of(a.n_pairs, a.E), flags, st);
}

cudaError_t expert_take_device_status(unsigned* flags) {
  unsigned tile = 0;
  cudaError_t e = expert_stream_take_status(flags);
  if (e == cudaSuccess) e = expert_tile_take_status(&tile);
  *flags |= tile;
  return e;
}

}  // namespace qlin
