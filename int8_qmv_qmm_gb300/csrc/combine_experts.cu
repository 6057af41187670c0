// The weighted sum of each token's experts (qlin.h has the definition).
//
// A thread takes 8 elements of a token's row (1, where rows do not start 16-byte
// aligned) and all of its experts: 2 bytes in for each expert's element, nothing used
// twice, so memory bounds it.

#include "device_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kThreads = 128;  // (256: 32 us for 30, 512: 43)

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Pack {
  T v[VEC];
};

// T: of out and add, Y: of the experts' rows.  (Nothing is __restrict__: what the preceding
// kernel writes while this one has started must not be taken for constant.)
template <typename T, typename Y, int VEC>
__global__ void __launch_bounds__(kThreads)
    combine_kernel(const Y* y, const int32_t* experts, const float* weights, const T* add,
                   int64_t add_stride, T* out, int64_t packs, int top_k, int64_t N) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t per_row = N / VEC;
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= packs) return;
  const int64_t t = i / per_row, n = (i - t * per_row) * VEC;
  float sum[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) sum[e] = 0.f;
  if (add) {
    const Pack<T, VEC> v = *reinterpret_cast<const Pack<T, VEC>*>(add + t * add_stride + n);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = widen(v.v[e]);
  }
  const Y* row = y + t * top_k * N + n;
  const int32_t* ex = experts + t * top_k;
  const float* wt = weights + t * top_k;
  // eight rows' loads before the first use of anything (also of rows without an expert,
  // which are then left out: waiting for the experts first took 41 us where this takes
  // 30, 4096 tokens of 8 rows of 2048)
  for (int j0 = 0; j0 < top_k; j0 += 8) {
    Pack<Y, VEC> v[8];
    float w[8];
    int e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = min(j0 + j, top_k - 1);
      v[j] = *reinterpret_cast<const Pack<Y, VEC>*>(row + at * N);
      w[j] = wt[at];
      e[j] = j0 + j < top_k ? ex[at] : -1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e[j] >= 0)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] = fmaf(w[j], widen(v[j].v[i]), sum[i]);
  }
  Pack<T, VEC> r;
#pragma unroll
  for (int e = 0; e < VEC; ++e) r.v[e] = Act<T>::from_f32_rn(sum[e]);
  *reinterpret_cast<Pack<T, VEC>*>(out + t * N + n) = r;
}

template <typename T, typename Y, int VEC>
void launch_t(const void* y, const int32_t* experts, const float* weights, const void* add,
              int64_t add_stride, void* out, int64_t T_, int top_k, int64_t N, unsigned flags,
              cudaStream_t st) {
  const int64_t packs = T_ * (N / VEC);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((packs + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, combine_kernel<T, Y, VEC>, static_cast<const Y*>(y), experts, weights,
                     static_cast<const T*>(add), add_stride, static_cast<T*>(out), packs, top_k,
                     N);
}

}  // namespace

qlin_status launch_combine_experts(const void* y, const int32_t* experts, const float* weights,
                                   const void* add, int64_t add_stride, void* out, int64_t T,
                                   int top_k, int64_t N, qlin_dtype dtype, qlin_dtype y_dtype,
                                   unsigned flags, cudaStream_t st) {
  auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool wide = N % 8 == 0 && add_stride % 8 == 0 && aligned(y) && aligned(add) && aligned(out);
  if (!wide && T * N > (int64_t(1) << 31) * kThreads)
    return fail(QLIN_ERR_UNSUPPORTED, "qlin_combine_experts: too many elements");
#define QLIN_COMBINE(T_, Y_)                                                                    \
  (wide ? launch_t<T_, Y_, 8>(y, experts, weights, add, add_stride, out, T, top_k, N, flags, st) \
        : launch_t<T_, Y_, 1>(y, experts, weights, add, add_stride, out, T, top_k, N, flags, st))
  if (dtype == QLIN_F16)
    y_dtype == QLIN_F32 ? QLIN_COMBINE(__half, float) : QLIN_COMBINE(__half, __half);
  else
    y_dtype == QLIN_F32 ? QLIN_COMBINE(__nv_bfloat16, float)
                        : QLIN_COMBINE(__nv_bfloat16, __nv_bfloat16);
#undef QLIN_COMBINE
  return check_launch("qlin_combine_experts");
}

}  // namespace qlin
