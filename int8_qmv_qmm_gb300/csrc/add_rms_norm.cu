// add_rms_norm: the residual's addition and the root-mean-square norm of the
// sum, one pass over the data.
//
//   h = x + residual                       (float32)
//   y = h * weight / sqrt(mean(h*h) + eps)
//
// A row is read once into registers, its sum of squares reduced over the
// threads that share it, and written once: 2 + r bytes in and 2 + r out for
// each element (r = 2 or 4, the residual's type), which is what bounds a call
// on many rows (8192 x 4096 bf16: 268 MB in 46 us, 5.8 TB/s with an event's
// overhead); a call on a few rows is a launch, two trips to memory and one
// reduction long (7 us).

#include <type_traits>

#include "device_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kMaxWidth = 32768;

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Pack {
  T v[VEC];
};

// One block per row.  VEC elements to a load (8 where every row starts 16-byte
// aligned, else 1), NV of them for each thread.
template <typename T, typename R, int VEC, int NV>
__global__ void __launch_bounds__(1024)
    add_rms_norm_kernel(const T* x, int64_t x_stride, const T* __restrict__ weight,
                        const R* residual, int64_t r_stride, R* residual_out, T* y, int K,
                        float eps) {
  __shared__ float partial[32];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * x_stride;
  grid_launch_dependents();
  grid_dependency_wait();
  float h[NV][VEC];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = (i * blockDim.x + threadIdx.x) * VEC;
    if (k < K) {
      const Pack<T, VEC> xv = *reinterpret_cast<const Pack<T, VEC>*>(xr + k);
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[i][e] = widen(xv.v[e]);
      if (residual) {
        const Pack<R, VEC> rv =
            *reinterpret_cast<const Pack<R, VEC>*>(residual + row * r_stride + k);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[i][e] += widen(rv.v[e]);
        if (residual_out) {
          Pack<R, VEC> ov;
#pragma unroll
          for (int e = 0; e < VEC; ++e) ov.v[e] = narrow<R>(h[i][e]);
          *reinterpret_cast<Pack<R, VEC>*>(residual_out + row * K + k) = ov;
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum += h[i][e] * h[i][e];
    }
  }
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = (threadIdx.x & 31) < warps ? partial[threadIdx.x & 31] : 0.f;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  }
  const float inv = 1.0f / sqrtf(sum / float(K) + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = (i * blockDim.x + threadIdx.x) * VEC;
    if (k < K) {
      const Pack<T, VEC> wv = *reinterpret_cast<const Pack<T, VEC>*>(weight + k);
      Pack<T, VEC> yv;
#pragma unroll
      for (int e = 0; e < VEC; ++e) yv.v[e] = narrow<T>(h[i][e] * inv * widen(wv.v[e]));
      *reinterpret_cast<Pack<T, VEC>*>(y + row * K + k) = yv;
    }
  }
}

template <typename T, typename R, int VEC, int NV>
void launch_t(const void* x, int64_t xs, const void* w, const void* r, int64_t rs, void* ro,
              void* y, int64_t M, int64_t K, float eps, unsigned flags, cudaStream_t st) {
  const int64_t packs = (K + VEC - 1) / VEC;
  const int64_t threads = ((packs + NV - 1) / NV + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(M));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, add_rms_norm_kernel<T, R, VEC, NV>, static_cast<const T*>(x), xs,
                     static_cast<const T*>(w), static_cast<const R*>(r), rs,
                     static_cast<R*>(ro), static_cast<T*>(y), int(K), eps);
}

template <typename T, typename R>
qlin_status dispatch(const void* x, int64_t xs, const void* w, const void* r, int64_t rs,
                     void* ro, void* y, int64_t M, int64_t K, float eps, unsigned flags,
                     cudaStream_t st) {
  auto aligned = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool wide = K % 8 == 0 && xs % 8 == 0 && rs % 8 == 0 && aligned(x) && aligned(w) &&
                    aligned(r) && aligned(ro) && aligned(y);
  // Loads of 8 where every row starts aligned (8192 x 1000 f16: 17 us, 33 with loads
  // of 1; 8192 x 4096 bf16: 46, 126).  Two of them a thread where there are rows enough
  // to fill the SMs (8192 x 4096: 46 us, 52 with one; 4096 x 8192: 48, 56; four: 50 and
  // 54), else one, which is a shorter way (32 x 4096 with a float32 residual: 7 us, 9);
  // one too where a row is a few warps' (8192 x 512: 13 us, 15).
  if (wide) {
    if (K <= 1024 || (K <= 8192 && M <= 4 * sm_count()))
      launch_t<T, R, 8, 1>(x, xs, w, r, rs, ro, y, M, K, eps, flags, st);
    else if (K <= 16384)
      launch_t<T, R, 8, 2>(x, xs, w, r, rs, ro, y, M, K, eps, flags, st);
    else
      launch_t<T, R, 8, 4>(x, xs, w, r, rs, ro, y, M, K, eps, flags, st);
  } else {  // (up to 4096 four a thread: 8192 x 2047 60 us, 91 with 32)
    if (K <= 4096)
      launch_t<T, R, 1, 4>(x, xs, w, r, rs, ro, y, M, K, eps, flags, st);
    else
      launch_t<T, R, 1, 32>(x, xs, w, r, rs, ro, y, M, K, eps, flags, st);
  }
  return check_launch("qlin_add_rms_norm");
}

}  // namespace

qlin_status launch_add_rms_norm(const void* x, int64_t x_stride, const void* weight,
                                const void* residual, int64_t residual_stride,
                                void* residual_out, void* y, int64_t M, int64_t K, float eps,
                                qlin_dtype dtype, qlin_dtype rdtype, unsigned flags,
                                cudaStream_t st) {
  static_assert(8 * 4 * 1024 >= kMaxWidth && 32 * 1024 >= kMaxWidth, "a row fits in a block");
  if (dtype == QLIN_F16)
    return rdtype == QLIN_F32
               ? dispatch<__half, float>(x, x_stride, weight, residual, residual_stride,
                                         residual_out, y, M, K, eps, flags, st)
               : dispatch<__half, __half>(x, x_stride, weight, residual, residual_stride,
                                          residual_out, y, M, K, eps, flags, st);
  return rdtype == QLIN_F32
             ? dispatch<__nv_bfloat16, float>(x, x_stride, weight, residual, residual_stride,
                                              residual_out, y, M, K, eps, flags, st)
             : dispatch<__nv_bfloat16, __nv_bfloat16>(x, x_stride, weight, residual,
                                                      residual_stride, residual_out, y, M, K,
                                                      eps, flags, st);
}

}  // namespace qlin
