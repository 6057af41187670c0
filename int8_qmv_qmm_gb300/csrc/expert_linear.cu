// The experts' products from packed weights (qlin.h has the definition): which kernel
// takes a call.

#include <cstdlib>

#include "expert_plan.cuh"
#include "qlin_internal.h"

namespace qlin {

namespace {

// Rows of an expert, were they spread evenly (the routing itself is on the device).
double rows_of(int64_t n_pairs, int E) {
  return double(n_pairs) / double(E < n_pairs ? E : n_pairs);
}

// Tiles of 8 tokens for the streaming kernel; 0: the tensor-core kernel.
int stream_tiles(int64_t n_pairs, int E, int64_t K) {
  const double rows = rows_of(n_pairs, E);
  double most = 32.0;
  if (const char* env = std::getenv("QLIN_EXPERT_MOST")) most = std::atof(env);
  return rows <= most ? expert_stream_tiles(K, rows) : 0;
}

}  // namespace

size_t expert_linear_workspace_size(int64_t n_pairs, int E, int64_t N, int64_t K) {
  return n_pairs > 0 && !stream_tiles(n_pairs, E, K) ? expert_tile_workspace_size(n_pairs, E, N, K)
                                                   : 0;
}

qlin_status launch_expert_linear(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st) {
  const int tiles = stream_tiles(a.n_pairs, a.E, a.K);
  if (tiles) return launch_expert_stream(a, bits, dtype, tiles, flags, st);
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
