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
// 8192 tokens, 8 of 256 experts by sigmoids with a bias out of 4 of 8 groups, take 24.8 us:
// 15 for the scores, 4 for the second launch's sums over the other CTAs' counts, 1 for its
// scan and 4 for placing.  The scores are bound by their instructions, about 1580 a token,
// which take 74% of the issue slots.  The second launch waits for what it loads (its warps
// issue a quarter of the time).  One token takes 4.8, the latency of its rounds.
//
// Scores and choices are float32, one rounding an operation, so that near ties fall
// the same way wherever the same operations are done.

#include <cmath>

#include "device_common.cuh"
#include "qlin_internal.h"

namespace qlin {
namespace {

// Warps of a CTA: as many as fit with their scratch.
template <int NE>
constexpr int kWarpsFor = NE == 16 ? 16 : 32;

// A warp's scratch holds an expert's value at spot(e): groups of 32 neighbours, read
// side by side, start in different banks.
__host__ __device__ constexpr int spot(int e) { return e + (e >> 5) * 4; }

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
  int32_t* counts;  // [CTAs][stride_of(E)] (more than one CTA)
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

// What a lane keeps over its tokens.
template <int NE>
struct Lane {
  float bias[NE];
  int group[NE];  // bit of each of its experts' groups among the groups that are kept
  int lanes;      // that share a group
};

// Leaves out the experts in groups that are not kept.  v: what a group's value is made
// of (-infinity: not eligible), through the warp's scratch.
template <int NE>
__device__ __forceinline__ void keep_groups(const Args& a, const Lane<NE>& own,
                                            const float (&v)[NE], float* scratch,
                                            uint32_t (&key)[NE]) {
  const int lane = threadIdx.x & 31, size = a.E / a.groups;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (lane + 32 * i < a.E) scratch[spot(lane + 32 * i)] = v[i];
  __syncwarp();
  const int lanes = own.lanes, g = lane / lanes;
  float v1 = -INFINITY, v2 = -INFINITY;
  if (g < a.groups) {
#pragma unroll 4
    for (int j = lane % lanes; j < size; j += lanes) {
      const float t = scratch[spot(g * size + j)];
      v2 = fmaxf(v2, fminf(v1, t));
      v1 = fmaxf(v1, t);
    }
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
  for (int i = 0; i < NE; ++i)
    if (!(kept >> own.group[i] & 1u)) key[i] = 0u;
}

template <typename T, int NE>
__device__ __forceinline__ void load_row(const Args& a, int64_t t, T (&x)[NE]) {
  const int lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(a.logits) + t * a.stride;
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (lane + 32 * i < a.E) x[i] = row[lane + 32 * i];
}

// Chooses token t's experts from its logits; lane j returns its j-th one (-1: none).
template <typename T, int NE>
__device__ int route_token(const Args& a, const Lane<NE>& own, int64_t t, const T (&raw)[NE],
                           float* scratch) {
  const int lane = threadIdx.x & 31;
  float x[NE], score[NE];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    x[i] = lane + 32 * i < a.E ? fmaxf(widen(raw[i]), -INFINITY) : -INFINITY;  // (NaN goes)
    top = fmaxf(top, x[i]);
  }
  const bool softmax = !a.sigmoid;
  // the scores' own sum, where a choice (which has to come out the same in any order
  // of summing: in 64 bits) or the weights need it
  float sum = 1.f;
  if (softmax) {
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
#pragma unroll
    for (int i = 0; i < NE; ++i) score[i] = x[i] == top ? 1.f : expf(x[i] - top);
    if (a.bias) {
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) z += x[i] > -INFINITY ? double(score[i]) : 0.0;
      for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(kAll, z, d);
      sum = float(z);
    } else if (!a.renormalise) {
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) sum += x[i] > -INFINITY ? score[i] : 0.f;
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) score[i] = __frcp_rn(__fadd_rn(1.f, expf(-x[i])));
  }
  uint32_t key[NE];
  float group_part[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    float choice = x[i];
    if (a.bias) {
      if (softmax) score[i] = __fdiv_rn(score[i], sum);
      choice = __fadd_rn(score[i], own.bias[i]);
    }
    key[i] = x[i] > -INFINITY ? key_of(choice) : 0u;
    group_part[i] = !key[i] ? -INFINITY : !a.bias && a.top2 ? score[i] : choice;
  }
  if (a.bias && softmax) sum = 1.f;  // (they are shares already)
  if (a.groups > 1) keep_groups<NE>(a, own, group_part, scratch, key);

  __syncwarp();
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (lane + 32 * i < a.E) scratch[spot(lane + 32 * i)] = score[i];
  int chosen = -1;
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t most = __reduce_max_sync(kAll, best);
    if (!most) break;
    const unsigned mine = best == most ? unsigned(lane + 32 * at) : ~0u;
    const unsigned e = __reduce_min_sync(kAll, mine);
    if (mine == e) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (i == at) key[i] = 0u;
    }
    if (lane == j) chosen = int(e);
  }
  __syncwarp();
  const float got = chosen >= 0 ? scratch[spot(chosen)] : 0.f;
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

// The sum of v over the threads before this one (all threads; buf: an int a warp).
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
// [WARPS][E + 1] of shared memory.  (Pairs without an expert count as expert E.)
template <int kWarps>
__device__ void place_pairs(const Args& a, int64_t p0, int64_t p1, const int* base, int* counts) {
  constexpr int kThreads = kWarps * 32;
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
    for (int w0 = 0; w0 < kWarps; w0 += 8) {
      int n[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) n[w] = counts[(w0 + w) * width + e];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        counts[(w0 + w) * width + e] = at;
        at += n[w];
      }
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

// Counts of a CTA in the workspace: whole vectors of four.
__host__ __device__ constexpr int stride_of(int E) { return (E + 4) / 4 * 4; }

__host__ __device__ constexpr int scratch_words(int E) {
  const int words = spot(E - 1) + 1;
  return words > E + 1 ? words : E + 1;
}

template <typename T, int NE>
__global__ void __launch_bounds__(kWarpsFor<NE> * 32) route_kernel(const Args a) {
  constexpr int kWarps = kWarpsFor<NE>, kThreads = kWarps * 32;
  // [kWarps][scratch]: the warps' groups and scores, later their counts; base [E + 1]
  extern __shared__ int shared[];
  __shared__ int buf[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int width = a.E + 1, words = scratch_words(a.E);
  int* base = shared + kWarps * words;
  for (int i = threadIdx.x; i < width; i += kThreads) base[i] = 0;
  Lane<NE> own;
  own.lanes = 32;
  while (own.lanes * a.groups > 32) own.lanes >>= 1;
  const int size = a.E / a.groups;
#pragma unroll
  for (int i = 0; i < NE; ++i) own.group[i] = min((lane + 32 * i) / size * own.lanes, 31);
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
#pragma unroll
  for (int i = 0; i < NE; ++i)
    own.bias[i] = a.bias && lane + 32 * i < a.E ? a.bias[lane + 32 * i] : 0.f;
  const int64_t t0 = blockIdx.x * a.per, t1 = min(t0 + a.per, a.T);
  T x[NE], next[NE];
  if (t0 + warp < t1) load_row<T, NE>(a, t0 + warp, next);
  for (int64_t t = t0 + warp; t < t1; t += kWarps) {
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] = next[i];
    if (t + kWarps < t1) load_row<T, NE>(a, t + kWarps, next);
    const int e =
        route_token<T, NE>(a, own, t, x, reinterpret_cast<float*>(shared) + warp * words);
    if (lane < a.top_k) atomicAdd(base + (e < 0 ? a.E : e), 1);
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < stride_of(a.E); e += kThreads)
      a.counts[int64_t(blockIdx.x) * stride_of(a.E) + e] = e < width ? base[e] : 0;
    return;
  }
  offsets_of(a, base, buf, true);
  place_pairs<kWarps>(a, 0, a.T * a.top_k, base, shared);
}

// The second launch, one CTA for each of the first's.
template <int kWarps>
__global__ void __launch_bounds__(kWarps * 32) place_kernel(const Args a) {
  constexpr int kThreads = kWarps * 32;
  extern __shared__ int shared[];
  __shared__ int buf[kWarps];
  const int width = a.E + 1;
  int* base = shared + kWarps * width;
  int* before = base + stride_of(a.E);  // of the pairs in the CTAs before this one
  for (int i = threadIdx.x; i < 2 * stride_of(a.E); i += kThreads) base[i] = 0;
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
  // four experts a load, the CTAs' counts over as many threads as there are
  const int vectors = stride_of(a.E) / 4, teams = kThreads / vectors;
  const int team = int(threadIdx.x) / vectors, v = int(threadIdx.x) % vectors;
  if (team < teams) {
    int4 all = make_int4(0, 0, 0, 0), first = all;
#pragma unroll 12
    for (int c = team; c < int(gridDim.x); c += teams) {
      const int4 n = reinterpret_cast<const int4*>(a.counts)[int64_t(c) * vectors + v];
      all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
      if (c < int(blockIdx.x)) first.x += n.x, first.y += n.y, first.z += n.z, first.w += n.w;
    }
    atomicAdd(base + 4 * v, all.x);
    atomicAdd(base + 4 * v + 1, all.y);
    atomicAdd(base + 4 * v + 2, all.z);
    atomicAdd(base + 4 * v + 3, all.w);
    atomicAdd(before + 4 * v, first.x);
    atomicAdd(before + 4 * v + 1, first.y);
    atomicAdd(before + 4 * v + 2, first.z);
    atomicAdd(before + 4 * v + 3, first.w);
  }
  __syncthreads();
  offsets_of(a, base, buf, blockIdx.x == 0);
  for (int e = threadIdx.x; e < width; e += kThreads) base[e] += before[e];
  __syncthreads();
  const int64_t t0 = blockIdx.x * a.per, t1 = min(t0 + a.per, a.T);
  place_pairs<kWarps>(a, t0 * a.top_k, t1 * a.top_k, base, shared);
}

// Tokens that one CTA takes with its warps: up to this many in one launch.
constexpr int64_t kOneCta = 32;
constexpr int64_t kTokensACta = 16;  // at least, in two launches
constexpr int kMostCtas = 1024;

template <typename T, int NE>
qlin_status launch_t(Args a, unsigned flags, cudaStream_t st) {
  constexpr int kWarps = kWarpsFor<NE>;
  int64_t ctas = 1;
  if (a.T > kOneCta) {
    const int64_t most = sm_count() < kMostCtas ? sm_count() : kMostCtas;
    ctas = (a.T + kTokensACta - 1) / kTokensACta;
    ctas = ctas < most ? ctas : most;
  }
  a.per = (a.T + ctas - 1) / ctas;
  if (ctas > 1) ctas = (a.T + a.per - 1) / a.per;
  static_assert((kWarpsFor<16> * scratch_words(512) + 513) * 4 <= 48 * 1024 - 256 &&
                    (kWarpsFor<8> * scratch_words(256) + 257) * 4 <= 48 * 1024 - 256 &&
                    (kWarpsFor<16> * 513 + 2 * 516) * 4 <= 48 * 1024 - 256 &&
                    (kWarpsFor<8> * 257 + 2 * 260) * 4 <= 48 * 1024 - 256,
                "without asking for more");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = size_t(kWarps * scratch_words(a.E) + a.E + 1) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, route_kernel<T, NE>, a) != cudaSuccess)
    return check_launch("qlin_route_experts");
  if (ctas > 1) {
    cfg.dynamicSmemBytes = size_t(kWarps * (a.E + 1) + 2 * stride_of(a.E)) * 4;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, place_kernel<kWarps>, a);
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
  // (for as many CTAs as any device takes: the size does not depend on it)
  const int64_t n = (T + kTokensACta - 1) / kTokensACta;
  return size_t(n < kMostCtas ? n : kMostCtas) * stride_of(E) * 4;
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
