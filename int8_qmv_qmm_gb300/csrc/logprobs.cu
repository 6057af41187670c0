// Log probabilities of given tokens, the entropy and the likeliest tokens of rows of
// logits (qlin.h has the definition).

#include <cmath>

#include "device_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

struct Args {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float* logprobs;
  float* entropy;
  int top;
  int32_t* top_tokens;
  float* top_logprobs;
  int64_t M;
  int V;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ uint32_t key_of(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (!key) return -INFINITY;
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const Args a) {
  __shared__ unsigned long long best_of[kWarps];
  __shared__ float sums[2][kWarps];
  __shared__ unsigned long long s_best;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t m = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* row = static_cast<const T*>(a.logits) + m * a.stride;
  // the elements in order: larger ones first, equal ones by index
  auto next = [&](unsigned long long below) {
    unsigned long long best = 0;
    for (int i = threadIdx.x; i < a.V; i += kThreads) {
      const uint32_t k = key_of(widen(row[i]));
      const unsigned long long v = k ? (unsigned long long)(k) << 32 | uint32_t(~i) : 0ull;
      if (v < below && v > best) best = v;
    }
    for (int d = 16; d; d >>= 1) {
      const unsigned long long o = __shfl_xor_sync(kAll, best, d);
      best = o > best ? o : best;
    }
    __syncthreads();
    if (lane == 0) best_of[warp] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) best = best_of[w] > best ? best_of[w] : best;
      s_best = best;
    }
    __syncthreads();
    return s_best;
  };
  const unsigned long long first = next(~0ull);
  const float top = value_of(uint32_t(first >> 32));
  float z = 0.f, u = 0.f;
  for (int i = threadIdx.x; i < a.V; i += kThreads) {
    const float v = widen(row[i]);
    if (!(v > -INFINITY)) continue;
    const float d = v == top ? 0.f : v - top, e = expf(d);
    z += e;
    if (e > 0.f) u += e * d;
  }
  for (int d = 16; d; d >>= 1) {
    z += __shfl_xor_sync(kAll, z, d);
    u += __shfl_xor_sync(kAll, u, d);
  }
  if (lane == 0) {
    sums[0][warp] = z;
    sums[1][warp] = u;
  }
  __syncthreads();
  z = u = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    z += sums[0][w];
    u += sums[1][w];
  }
  const float log_z = logf(z);
  auto logprob = [&](float v) {
    if (!(v > -INFINITY)) return -INFINITY;
    return (v == top ? 0.f : v - top) - log_z;
  };
  if (threadIdx.x == 0) {
    const int t = a.tokens[m];
    a.logprobs[m] = t >= 0 && t < a.V ? logprob(widen(row[t])) : -INFINITY;
    a.entropy[m] = first ? log_z - u / z : 0.f;
  }
  unsigned long long at = first;
  for (int j = 0; j < a.top; ++j) {
    if (j) at = at ? next(at) : 0ull;
    if (threadIdx.x == 0) {
      a.top_tokens[m * a.top + j] = at ? int32_t(~uint32_t(at)) : -1;
      a.top_logprobs[m * a.top + j] = at ? logprob(value_of(uint32_t(at >> 32))) : -INFINITY;
    }
  }
}

template <typename T>
void launch_t(const Args& a, unsigned flags, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.M));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a);
}

}  // namespace

qlin_status launch_token_logprobs(const void* logits, int64_t stride, const int32_t* tokens,
                                  float* logprobs, float* entropy, int top, int32_t* top_tokens,
                                  float* top_logprobs, int64_t M, int64_t V, qlin_dtype ldtype,
                                  unsigned flags, cudaStream_t st) {
  const Args a = {logits, stride, tokens, logprobs, entropy, top, top_tokens, top_logprobs, M,
                  int(V)};
  if (ldtype == QLIN_F32)
    launch_t<float>(a, flags, st);
  else if (ldtype == QLIN_F16)
    launch_t<__half>(a, flags, st);
  else
    launch_t<__nv_bfloat16>(a, flags, st);
  return check_launch("qlin_token_logprobs");
}

}  // namespace qlin
