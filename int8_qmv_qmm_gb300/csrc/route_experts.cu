// Routing of tokens to experts, and the plan that groups their rows (qlin.h has the
// definition).
//
// One warp scores a token: a lane holds every 32nd expert's logit, so the row is read
// once, and the top-k are k rounds of a warp-wide maximum over order-preserving bit
// patterns, the lowest index first among equal ones.  The plan is a counting sort of
// the pairs by expert that keeps their order: every CTA counts the experts of its own
// stretch of tokens, a second launch (the same one, where one CTA has all tokens) adds
// up what lies before each stretch and expert and places the pairs.
//
// Scores and choices are float32, one rounding an operation, so that near ties fall
// the same way wherever the same operations are done.

#include <cmath>

#include "device_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxExperts = 512;
static_assert(kMaxExperts <= kThreads, "a thread for each expert in the scans");

struct Args {
  const void* logits;
  int64_t stride;
  const float* bias;
  int sigmoid, groups, top_groups, top2, top_k, renormalise;
  float scale;
  int32_t* experts;
  float* weights;
  int32_t* order;
  int32_t* offsets;
  int32_t* counts;  // [CTAs][E + 1] (more than one CTA)
  int64_t T;
  int E;
  int64_t per;  // tokens of a CTA
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// Bits that order as the numbers do; 0 for what cannot be chosen (-infinity, NaN).
__device__ __forceinline__ uint32_t key_of(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.f);  // (-0 becomes 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr unsigned kAll = 0xffffffffu;

// Whether each of a lane's experts is in a group that is kept.  v: what a group's
// value is made of (-infinity: not eligible), through the warp's scratch.
template <int NE>
__device__ __forceinline__ void keep_groups(const Args& a, const float (&v)[NE], float* scratch,
                                            uint32_t (&key)[NE]) {
  const int lane = threadIdx.x & 31, size = a.E / a.groups;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (lane + 32 * i < a.E) scratch[lane + 32 * i] = v[i];
  __syncwarp();
  int lanes = 32;  // that share a group
  while (lanes * a.groups > 32) lanes >>= 1;
  const int g = lane / lanes;
  float v1 = -INFINITY, v2 = -INFINITY;
  if (g < a.groups)
    for (int j = lane % lanes; j < size; j += lanes) {
      const float t = scratch[g * size + j];
      v2 = fmaxf(v2, fminf(v1, t));
      v1 = fmaxf(v1, t);
    }
  for (int d = lanes / 2; d; d >>= 1) {
    const float o1 = __shfl_xor_sync(kAll, v1, d), o2 = __shfl_xor_sync(kAll, v2, d);
    v2 = fmaxf(fmaxf(v2, o2), fminf(v1, o1));
    v1 = fmaxf(v1, o1);
  }
  const uint32_t mine =
      g < a.groups ? key_of(a.top2 && v2 > -INFINITY ? __fadd_rn(v1, v2) : v1) : 0u;
  int better = 0;
  for (int o = 0; o < a.groups; ++o) {
    const uint32_t other = __shfl_sync(kAll, mine, o * lanes);
    better += other > mine || (other == mine && o < g);
  }
  const unsigned kept = __ballot_sync(kAll, g < a.groups && better < a.top_groups);
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 32 * i;
    if (e < a.E && !(kept >> (e / size * lanes) & 1u)) key[i] = 0u;
  }
}

// Chooses token t's experts; lane j returns its j-th one (-1: none).
template <typename T, int NE>
__device__ int route_token(const Args& a, int64_t t, float* scratch) {
  const int lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(a.logits) + t * a.stride;
  float x[NE], score[NE];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < a.E ? widen(row[e]) : -INFINITY;
    x[i] = fmaxf(x[i], -INFINITY);  // (-infinity for NaN)
    top = fmaxf(top, x[i]);
  }
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
  const bool softmax = !a.sigmoid;
  if (softmax) {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      score[i] = x[i] == top ? 1.f : expf(x[i] - top);
    // (no row of -infinity alone comes here with x == top and a use for its score)
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) score[i] = __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x[i])));
  }
  uint32_t key[NE];
  float group_part[NE];
  // the scores' own sum, where a choice (which has to come out the same in any order
  // of summing: in 64 bits) or the weights need it
  float sum = 1.f;
  if (softmax && a.bias) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i) z += x[i] > -INFINITY ? double(score[i]) : 0.0;
    for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(kAll, z, d);
    sum = float(z);
  } else if (softmax && !a.renormalise) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) sum += x[i] > -INFINITY ? score[i] : 0.f;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 32 * i;
    float choice = x[i];
    if (a.bias) {
      if (softmax) score[i] = __fdiv_rn(score[i], sum);
      choice = e < a.E ? __fadd_rn(score[i], a.bias[e]) : -INFINITY;
    }
    key[i] = x[i] > -INFINITY ? key_of(choice) : 0u;
    group_part[i] = !key[i] ? -INFINITY : !a.bias && a.top2 ? score[i] : choice;
  }
  if (a.bias && softmax) sum = 1.f;  // (they are shares already)
  if (a.groups > 1) keep_groups<NE>(a, group_part, scratch, key);

  int chosen = -1;
  float got = 0.f;
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t best = 0u;
    int at = 0;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
        s = score[i];
      }
    const uint32_t most = __reduce_max_sync(kAll, best);
    if (!most) break;
    const unsigned e = __reduce_min_sync(kAll, best == most ? unsigned(lane + 32 * at) : ~0u);
    const int owner = int(e & 31u);
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane == owner && i == int(e >> 5)) key[i] = 0u;
    s = __shfl_sync(kAll, s, owner);
    if (lane == j) {
      chosen = int(e);
      got = s;
    }
  }
  if (a.renormalise) {
    sum = got;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  }
  if (lane < a.top_k) {
    const float w = got > 0.f ? __fdiv_rn(got, sum) * a.scale : 0.f;
    a.experts[t * a.top_k + lane] = chosen;
    a.weights[t * a.top_k + lane] = w;
  }
  return chosen;
}

// The sum of v over the threads before this one (all threads; buf: kWarps ints).
__device__ __forceinline__ int scan_before(int v, int* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = v;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) buf[warp] = upto;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += buf[w];
  __syncthreads();
  return before + upto - v;
}

// Writes the order of the pairs [p0, p1): a pair's place is base[its expert] + the
// number of pairs of that expert before it.  Each warp takes a stretch of its own,
// counts its experts, and goes on from what the warps before it have.  counts:
// [kWarps][E + 1] of shared memory.  (Pairs without an expert count as expert E.)
__device__ void place_pairs(const Args& a, int64_t p0, int64_t p1, const int* base, int* counts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int width = a.E + 1;
  for (int i = threadIdx.x; i < kWarps * width; i += kThreads) counts[i] = 0;
  __syncthreads();
  const int64_t each = ((p1 - p0 + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int64_t w0 = min(p0 + warp * each, p1), w1 = min(w0 + each, p1);
  int* mine = counts + warp * width;
  auto expert_of = [&](int64_t p) {
    const int e = p < w1 ? a.experts[p] : a.E;
    return e < 0 ? a.E : e;
  };
  for (int64_t p = w0 + lane; p - lane < w1; p += 32) {
    const int e = expert_of(p);
    const unsigned live = __ballot_sync(kAll, p < w1);
    const unsigned same = __match_any_sync(kAll, e) & live;
    if (p < w1 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < width; e += kThreads) {
    int at = base[e];
    for (int w = 0; w < kWarps; ++w) {
      const int n = counts[w * width + e];
      counts[w * width + e] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t p = w0 + lane; p - lane < w1; p += 32) {
    const int e = expert_of(p);
    const unsigned live = __ballot_sync(kAll, p < w1);
    const unsigned same = __match_any_sync(kAll, e) & live;
    int at = 0;
    if (p < w1) at = mine[e];
    __syncwarp();
    if (p < w1) {
      a.order[at + __popc(same & ((1u << lane) - 1u))] = int32_t(p);
      if (lane == __ffs(same) - 1) mine[e] = at + __popc(same);
    }
    __syncwarp();
  }
}

// offsets (the first CTA's to write) and, in base, what comes before each expert;
// in: base holds the number of pairs of each expert (E + 1).
__device__ void offsets_of(const Args& a, int* base, int* buf, bool write) {
  const int e = threadIdx.x;
  // (E can be as many as the threads: expert E, the pairs without one, comes after all)
  const int before = scan_before(e < a.E ? base[e] : 0, buf);
  const int last = e == a.E - 1 ? before + base[e] : 0;
  __syncthreads();
  if (e < a.E) base[e] = before;
  if (e == a.E - 1) base[a.E] = last;
  if (write && e < a.E) a.offsets[e] = before;
  if (write && e == a.E - 1) a.offsets[a.E] = last;
  __syncthreads();
}

template <typename T, int NE>
__global__ void __launch_bounds__(kThreads) route_kernel(const Args a) {
  // [kWarps][E + 1] words: the warps' groups, later their counts; base [E + 1]
  extern __shared__ int shared[];
  __shared__ int buf[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int width = a.E + 1;
  int* base = shared + kWarps * width;
  for (int i = threadIdx.x; i < width; i += kThreads) base[i] = 0;
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t t0 = blockIdx.x * a.per, t1 = min(t0 + a.per, a.T);
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
    const int e = route_token<T, NE>(a, t, reinterpret_cast<float*>(shared) + warp * width);
    if (lane < a.top_k) atomicAdd(base + (e < 0 ? a.E : e), 1);
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < width; e += kThreads)
      a.counts[int64_t(blockIdx.x) * width + e] = base[e];
    return;
  }
  offsets_of(a, base, buf, true);
  place_pairs(a, 0, a.T * a.top_k, base, shared);
}

// The second launch, one CTA for each of the first's.
__global__ void __launch_bounds__(kThreads) place_kernel(const Args a) {
  extern __shared__ int shared[];
  __shared__ int buf[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int width = a.E + 1;
  int* base = shared + kWarps * width;
  int* before = base + width;  // of the pairs in the CTAs before this one
  for (int i = threadIdx.x; i < 2 * width; i += kThreads) base[i] = 0;
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
  for (int e = lane; e < width; e += 32) {
    int all = 0, first = 0;
#pragma unroll 4
    for (int c = warp; c < int(gridDim.x); c += kWarps) {
      const int n = a.counts[int64_t(c) * width + e];
      all += n;
      first += c < int(blockIdx.x) ? n : 0;
    }
    atomicAdd(base + e, all);
    atomicAdd(before + e, first);
  }
  __syncthreads();
  offsets_of(a, base, buf, blockIdx.x == 0);
  for (int e = threadIdx.x; e < width; e += kThreads) base[e] += before[e];
  __syncthreads();
  const int64_t t0 = blockIdx.x * a.per, t1 = min(t0 + a.per, a.T);
  place_pairs(a, t0 * a.top_k, t1 * a.top_k, base, shared);
}

// Tokens that one CTA takes with its warps: up to this many in one launch.
constexpr int64_t kOneCta = 4 * kWarps;

int64_t ctas_for(int64_t T, int sms) {
  if (T <= kOneCta) return 1;
  const int64_t n = (T + kWarps - 1) / kWarps;
  return n < sms ? n : sms;
}

template <typename T, int NE>
qlin_status launch_t(Args a, unsigned flags, cudaStream_t st) {
  int64_t ctas = ctas_for(a.T, sm_count());
  a.per = (a.T + ctas - 1) / ctas;
  if (ctas > 1) ctas = (a.T + a.per - 1) / a.per;
  static_assert((kWarps + 2) * (kMaxExperts + 1) * 4 <= 40 * 1024, "without asking for more");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(kWarps + 2) * (a.E + 1) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, route_kernel<T, NE>, a) != cudaSuccess)
    return check_launch("qlin_route_experts");
  if (ctas > 1) {
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, place_kernel, a);
  }
  return check_launch("qlin_route_experts");
}

template <typename T>
qlin_status dispatch(const Args& a, unsigned flags, cudaStream_t st) {
  if (a.E <= 32) return launch_t<T, 1>(a, flags, st);
  if (a.E <= 64) return launch_t<T, 2>(a, flags, st);
  if (a.E <= 128) return launch_t<T, 4>(a, flags, st);
  if (a.E <= 256) return launch_t<T, 8>(a, flags, st);
  return launch_t<T, 16>(a, flags, st);
}

}  // namespace

size_t route_experts_workspace_size(int64_t T, int E) {
  if (T <= kOneCta) return 0;
  const int64_t n = (T + kWarps - 1) / kWarps;
  // (at most one CTA for each of 1024 SMs: the size does not depend on the device)
  return size_t(n < 1024 ? n : 1024) * (E + 1) * 4;
}

qlin_status launch_route_experts(const RouteArgs& r, void* workspace, unsigned flags,
                                 cudaStream_t st) {
  Args a = {};
  a.logits = r.logits;
  a.stride = r.stride;
  a.bias = r.bias;
  a.sigmoid = r.scoring == QLIN_SIGMOID;
  a.groups = r.groups;
  a.top_groups = r.top_groups;
  a.top2 = r.group_score == QLIN_GROUP_TOP2;
  a.top_k = r.top_k;
  a.renormalise = r.renormalise;
  a.scale = r.scale;
  a.experts = r.experts;
  a.weights = r.weights;
  a.order = r.order;
  a.offsets = r.offsets;
  a.counts = static_cast<int32_t*>(workspace);
  a.T = r.T;
  a.E = r.E;
  if (r.dtype == QLIN_F32) return dispatch<float>(a, flags, st);
  return r.dtype == QLIN_F16 ? dispatch<__half>(a, flags, st)
                             : dispatch<__nv_bfloat16>(a, flags, st);
}

}  // namespace qlin
