// The experts' products from packed weights (qlin.h has the definition).
//
// A warp takes one row of an expert's weights and up to 8 of the expert's tokens at a
// time; its lanes take the row's words in turn.

#include "device_common.cuh"
#include "expert_plan.cuh"
#include "qlin_internal.h"

namespace qlin {

__device__ unsigned int g_expert_status = 0;

namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 8;

template <int BITS, typename AT>
__global__ void __launch_bounds__(kWarps * 32) expert_kernel(const ExpertArgs a) {
  constexpr int kCodes = 32 / BITS;
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t n = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int expert = blockIdx.y;
  if (n >= a.N) return;
  const ExpertRows r = expert_rows(a, expert);
  if (r.bad && lane == 0) atomicOr(&g_expert_status, 1u);
  const int words = int(a.K) / kCodes, groups = int(a.K) / kGroup;
  const int64_t row = expert * a.N + n;
  const uint32_t* wq = a.wq + row * words;
  const AT* sc = static_cast<const AT*>(a.scales) + row * groups;
  const AT* bi = static_cast<const AT*>(a.biases) + row * groups;
  for (int i0 = 0; i0 < r.n; i0 += kTokens) {
    float acc[kTokens];
    const AT* x[kTokens];
    int64_t pair[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      acc[i] = 0.f;
      pair[i] = i0 + i < r.n ? a.order[r.first + i0 + i] : -1;
      if (pair[i] >= a.n_pairs || (i0 + i < r.n && pair[i] < 0)) {
        if (lane == 0) atomicOr(&g_expert_status, 1u);
        pair[i] = -1;
      }
      x[i] = static_cast<const AT*>(a.x) + (pair[i] < 0 ? 0 : pair[i] / a.pairs_per_row) * a.x_stride;
    }
    for (int w = lane; w < words; w += 32) {
      const uint32_t word = wq[w];
      const float s = Act<AT>::to_f32(sc[w * kCodes / kGroup]);
      const float b = Act<AT>::to_f32(bi[w * kCodes / kGroup]);
#pragma unroll
      for (int c = 0; c < kCodes; ++c) {
        const float v = fmaf(float(word >> (BITS * c) & ((1u << BITS) - 1u)), s, b);
#pragma unroll
        for (int i = 0; i < kTokens; ++i)
          if (pair[i] >= 0) acc[i] = fmaf(v, Act<AT>::to_f32(x[i][w * kCodes + c]), acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      for (int d = 16; d; d >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
      if (lane == 0 && pair[i] >= 0) {
        if (a.y_f32)
          static_cast<float*>(a.y)[pair[i] * a.N + n] = acc[i];
        else
          static_cast<AT*>(a.y)[pair[i] * a.N + n] = Act<AT>::from_f32_rn(acc[i]);
      }
    }
  }
}

template <int BITS, typename AT>
void launch_t(const ExpertArgs& a, unsigned flags, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.N + kWarps - 1) / kWarps), unsigned(a.E));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, expert_kernel<BITS, AT>, a);
}

}  // namespace

qlin_status launch_expert_linear(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st) {
  if (dtype == QLIN_F16)
    bits == 4 ? launch_t<4, __half>(a, flags, st) : launch_t<8, __half>(a, flags, st);
  else
    bits == 4 ? launch_t<4, __nv_bfloat16>(a, flags, st)
              : launch_t<8, __nv_bfloat16>(a, flags, st);
  return check_launch("qlin_expert_linear");
}

cudaError_t expert_take_device_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_expert_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_expert_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace qlin
