// The experts' products from packed weights (qlin.h has the definition): which kernel
// takes a call.

#include "expert_plan.cuh"
#include "qlin_internal.h"

namespace qlin {

qlin_status launch_expert_linear(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st) {
  // rows of an expert, were they spread evenly (the routing itself is on the device)
  const double rows = double(a.n_pairs) / double(a.E < a.n_pairs ? a.E : a.n_pairs);
  const int tiles = expert_stream_tiles(a.K, rows);
  return launch_expert_stream(a, bits, dtype, tiles, flags, st);
}

cudaError_t expert_take_device_status(unsigned* flags) {
  return expert_stream_take_status(flags);
}

}  // namespace qlin
