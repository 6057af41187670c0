// The experts' products from packed weights (qlin.h has the definition): which kernel
// takes a call.

#include <cstdlib>

#include "expert_plan.cuh"
#include "qlin_internal.h"

namespace qlin {

qlin_status launch_expert_linear(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st) {
  // rows of an expert, were they spread evenly (the routing itself is on the device)
  const double rows = double(a.n_pairs) / double(a.E < a.n_pairs ? a.E : a.n_pairs);
  const int tiles = expert_stream_tiles(a.K, rows);
  double most = 16.0;
  if (const char* env = std::getenv("QLIN_EXPERT_MOST")) most = std::atof(env);
  if (tiles && rows <= most) return launch_expert_stream(a, bits, dtype, tiles, flags, st);
  return launch_expert_tile(a, bits, dtype, rows, flags, st);
}

cudaError_t expert_take_device_status(unsigned* flags) {
  unsigned tile = 0;
  cudaError_t e = expert_stream_take_status(flags);
  if (e == cudaSuccess) e = expert_tile_take_status(&tile);
  *flags |= tile;
  return e;
}

}  // namespace qlin
