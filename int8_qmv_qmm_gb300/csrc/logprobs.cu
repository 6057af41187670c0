// Log probabilities of given tokens, the entropy and the likeliest tokens of rows of
// logits (qlin.h has the definition), in one pass over a row.
//
// A thread takes every T-th 16 bytes of the row (of a part of it, where a cluster of CTAs
// shares a row) and keeps, in float32, its largest logit m and where it stands, a
// reference c <= m, and sums over its logits of e = exp(x - c) and of e * (x - c): with
// the row's largest logit M they become Z and the entropy's mean.  The reference moves
// only where a logit passes it by 60, so that no sum is rescaled on the way, and x - c is
// a difference of the logits themselves: an exponential's error does not grow with them.
//
// The likeliest n tokens lie with the n threads whose largest logits are the largest, in
// the order of logits and indices: were one with another thread, the n threads' best
// would all come before it.  So those n threads' logits are looked over again (a few
// thousand bytes, in L2), the ones that come before the n-th thread's best are listed,
// and a listed one's place is the number of better ones.
//
// Logits of -infinity, NaN and the types' lowest values count as `lowest` on the way, of
// exponential 0.  Where that does not do (a part whose largest logit is near it, above
// 1e37 or infinite, fewer than n threads with a logit above it) a second, slower way takes
// the part: the definition, logit by logit.
//
// Exponentials are the hardware's (2 ulp): outputs are off by 3e-8 to 1.1e-7 of their size,
// over a set of rows.
//
// 2048 rows of 128256 in 16 bits, with the 5 likeliest, take 102 us, 5.2 TB/s: the
// instructions for an exponential and two sums of each logit take about as long as reading
// it.  One row of float32 with the 20 likeliest takes 10 us: launch, two rounds of loads,
// and a chain of exchanges in the CTAs and between the eight of the cluster.

#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "qlin_internal.h"
#include "sm100_ptx.cuh"

namespace qlin {
namespace {

// Of a CTA: four or five of them to an SM, so that one picks while others read.  (16-bit
// logits with four: 111 us for 102; float32 with five: 101 for 97.)
constexpr int kThreads = 256;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 1024;  // logits that are ranked by counting
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
using u64 = unsigned long long;

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

// Bits that order as the numbers do; 0 for what has no share (-infinity, NaN).
__device__ __forceinline__ uint32_t key_of(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.f);  // (-0 becomes 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (!key) return -INFINITY;
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ u64 place_of(float v, int index) {
  const uint32_t k = key_of(v);
  return k ? u64(k) << 32 | uint32_t(~index) : 0ull;
}

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ u64 warp_max(u64 v) {
  const uint32_t hi = __reduce_max_sync(kAll, uint32_t(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
  return u64(hi) << 32 | lo;
}

// What a logit that has no share counts as, and the largest logit below which that is
// not far enough away.
template <typename T>
struct Bounds {
  static constexpr float kLowest = -1e30f, kLow = -1e29f;
};
template <>
struct Bounds<__half> {
  static constexpr float kLowest = -65504.f, kLow = -60000.f;
};
constexpr float kHigh = 1e37f;

// 16 bytes of logits, none below kLowest, as pairs; and the largest.
template <typename T>
struct Pack {
  static constexpr int kElems = 16 / sizeof(T);
  float2 v[kElems / 2];
  float most;
};
template <typename T>
__device__ __forceinline__ Pack<T> clean(uint4 raw) {
  Pack<T> r;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (std::is_same<T, float>::value) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = fmaxf(__uint_as_float(w[i]), Bounds<T>::kLowest);
    r.v[0] = make_float2(f[0], f[1]);
    r.v[1] = make_float2(f[2], f[3]);
    r.most = fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
  } else {
    using T2 = typename Act<T>::T2;
    T2 low;
    low.x = low.y = Act<T>::from_f32_rn(Bounds<T>::kLowest);
    T2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __hmax2(*reinterpret_cast<const T2*>(&w[i]), low);
    const T2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    r.most = fmaxf(Act<T>::to_f32(m.x), Act<T>::to_f32(m.y));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        r.v[i] = __half22float2(h[i]);
      } else {
        const uint32_t b = *reinterpret_cast<const uint32_t*>(&h[i]);
        r.v[i] = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
      }
    }
  }
  return r;
}

// A CTA's part of a row, in 16-byte vectors on the memory's own boundaries: vector k is
// elements k * kElems - shift .., of which those in [0, n) are the row's.
template <typename T>
struct Part {
  static constexpr int kElems = 16 / sizeof(T);
  const T* row;
  int n, shift;
  int first, end;  // vectors

  __device__ __forceinline__ bool whole(int k) const {
    return k * kElems >= shift && (k + 1) * kElems - shift <= n;
  }
  __device__ __forceinline__ uint4 load(int k) const {
    // (not by the read-only path: the preceding kernel may have written them since the start)
    if (whole(k)) return *reinterpret_cast<const uint4*>(row + (k * kElems - shift));
    // an edge: what is not the row's counts as -infinity
    constexpr uint32_t kNone = std::is_same<T, float>::value    ? 0xff800000u
                               : std::is_same<T, __half>::value ? 0xfc00fc00u
                                                                : 0xff80ff80u;
    uint32_t w[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
    for (int e = 0; e < kElems; ++e) {
      const int i = k * kElems - shift + e;
      if (i >= 0 && i < n) {
        if constexpr (std::is_same<T, float>::value) {
          w[e] = __float_as_uint(row[i]);
        } else {
          const uint32_t b = *reinterpret_cast<const uint16_t*>(row + i);
          w[e / 2] = e % 2 ? (w[e / 2] & 0xffffu) | b << 16 : (w[e / 2] & 0xffff0000u) | b;
        }
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // f(value, index) for every logit of vector k
  template <class F>
  __device__ __forceinline__ void each(int k, F f) const {
    const uint4 raw = load(k);
    const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int e = 0; e < kElems; ++e) f(widen(t[e]), k * kElems - shift + e);
  }
};

struct Shared {
  static constexpr int kWarps = kThreads / 32;
  float red[3][kWarps];
  u64 sorted[kWarps][32];    // the threads' largest logits and their vectors
  int chosen[kMaxTop];       // threads
  int n_list;
  u64 last;                  // the last chosen one's
  u64 warp_best[kWarps];
  u64 list[kList];
  u64 best[kMaxTop];         // the part's likeliest, in order
  // of the cluster's CTAs (rank 0's are used)
  float sums[kMaxCluster][3];
  u64 all[kMaxCluster][kMaxTop];
};

template <class Op>
__device__ __forceinline__ float block_reduce(float v, float* buf, Op op) {
  for (int d = 16; d; d >>= 1) v = op(v, __shfl_xor_sync(kAll, v, d));
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v = op(v, buf[w]);
  return v;
}

// The part's likeliest `top` logits, one after another (the slower way).
template <typename T>
__device__ void pick_slowly(const Part<T>& part, int top, Shared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 mine = 0;
  for (int k = part.first + int(threadIdx.x); k < part.end; k += kThreads)
    part.each(k, [&](float v, int i) {
      const u64 p = place_of(v, i);
      mine = p > mine ? p : mine;
    });
  for (int j = 0; j < top; ++j) {
    const u64 w = warp_max(mine);
    __syncthreads();
    if (lane == 0) s.warp_best[warp] = w;
    __syncthreads();
    u64 best = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) best = s.warp_best[i] > best ? s.warp_best[i] : best;
    if (threadIdx.x == 0) s.best[j] = best;
    if (!best) continue;
    const int k = (int(~uint32_t(best)) + part.shift) / Part<T>::kElems;
    const int owner = (k - part.first) % kThreads;
    if (warp == owner / 32) {  // its warp looks for its next one
      u64 next = 0;
      for (int v = part.first + owner + kThreads * lane; v < part.end; v += kThreads * 32)
        part.each(v, [&](float x, int i) {
          const u64 p = place_of(x, i);
          if (p < best && p > next) next = p;
        });
      next = warp_max(next);
      if (lane == owner % 32) mine = next;
    }
  }
  __syncthreads();
}

// Sorts a warp's values, the largest to lane 0.
__device__ __forceinline__ u64 warp_sort(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size / 2; d; d >>= 1) {
      const u64 o = __shfl_xor_sync(kAll, v, d);
      // (the larger one to the lower lane in the stretches that descend)
      const bool larger = ((lane & d) == 0) == ((lane & size) == 0 || size == 32);
      v = (o > v) == larger ? o : v;
    }
  return v;
}

// How many of a list's first n values, in falling order, are larger than v.
__device__ __forceinline__ int larger_in(const u64* list, int n, u64 v) {
  int low = 0;
  for (int d = 32; d; d >>= 1)
    if (low + d <= n && list[low + d - 1] > v) low += d;
  return low;
}

// The part's likeliest `top` logits from the threads that have them; false where fewer
// threads have a logit to speak of, or the logits to rank are too many.
//
// The threads' best ones are sorted in each warp, and ranked by a search in each other
// warp's list.  (One warp picking the best of all, `top` times: 2048 rows with their
// first 5 took 119 us, with 20 172, where this took 111 and 127; without any, 97.)
template <typename T>
__device__ bool pick(const Part<T>& part, int top, float most, int at, Shared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 mine = warp_sort(
      most > Bounds<T>::kLowest ? u64(key_of(most)) << 32 | uint32_t(~at) : 0ull);
  s.sorted[warp][lane] = mine;
  if (threadIdx.x == 0) {
    s.n_list = 0;
    s.last = 0;
  }
  __syncthreads();
  if (lane < top && mine) {
    int rank = lane;
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i)
      rank += larger_in(s.sorted[(warp + i) % (kThreads / 32)], top, mine);
    if (rank < top) s.chosen[rank] = (int(~uint32_t(mine)) - part.first) % kThreads;
    if (rank == top - 1) s.last = mine;
  }
  __syncthreads();
  const u64 last = s.last;
  if (!last) return false;
  const float last_value = value_of(uint32_t(last >> 32));
  const int last_at = int(~uint32_t(last));
  for (int j = warp; j < top; j += kThreads / 32) {
    for (int k = part.first + s.chosen[j] + kThreads * lane; k < part.end; k += kThreads * 32) {
      if (clean<T>(part.load(k)).most < last_value) continue;
      part.each(k, [&](float v, int i) {
        if (v > last_value || (v == last_value && k <= last_at)) {
          const int n = atomicAdd(&s.n_list, 1);
          if (n < kList) s.list[n] = place_of(v, i);
        }
      });
    }
  }
  __syncthreads();
  const int n = s.n_list;
  if (n > kList) return false;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const u64 p = s.list[i];
    int better = 0;
    for (int j = 0; j < n; ++j) better += s.list[j] > p;
    if (better < top) s.best[better] = p;
  }
  __syncthreads();
  return true;
}

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4)
    logprobs_kernel(const Args a, int ranks) {
  __shared__ Shared s;
  constexpr int kElems = Part<T>::kElems, kUnroll = 4;
  const int rank = ranks > 1 ? int(ptx::cluster_ctarank()) : 0;
  const int64_t m = int64_t(blockIdx.x) / ranks;
  Part<T> part;
  part.row = static_cast<const T*>(a.logits) + m * a.stride;
  part.n = a.V;
  part.shift = int(reinterpret_cast<uintptr_t>(part.row) % 16 / sizeof(T));
  const int vectors = (a.V + part.shift + kElems - 1) / kElems;
  part.first = int(int64_t(vectors) * rank / ranks);
  part.end = int(int64_t(vectors) * (rank + 1) / ranks);
  grid_launch_dependents();
  grid_dependency_wait();
  if (ranks > 1) ptx::cluster_arrive_relaxed();  // (waited for before the first store to a peer)

  // the thread's logits
  float most = Bounds<T>::kLowest, c = Bounds<T>::kLowest;
  int at = 0;
  float2 sum = make_float2(0.f, 0.f), mean = make_float2(0.f, 0.f);
  auto take = [&](uint4 raw, int k) {
    const Pack<T> p = clean<T>(raw);
    if (p.most > c + 60.f) {
      // (where f is 0 what there was is gone: its product with d could have overflown)
      const float d = (c - p.most) * kLog2e, f = exp2_fast(d);
      mean.x = f > 0.f ? (mean.x + sum.x * d) * f : 0.f;
      mean.y = f > 0.f ? (mean.y + sum.y * d) * f : 0.f;
      sum.x *= f;
      sum.y *= f;
      c = p.most;
    }
    if (p.most > most) {
      most = p.most;
      at = k;
    }
    const float2 minus_c = make_float2(-c, -c), scale = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < kElems / 2; ++i) {
      const float2 d = __fmul2_rn(__fadd2_rn(p.v[i], minus_c), scale);
      const float2 e = make_float2(exp2_fast(d.x), exp2_fast(d.y));
      sum = __fadd2_rn(sum, e);
      mean = __ffma2_rn(e, d, mean);
    }
  };
  int k = part.first + int(threadIdx.x);
  for (; k + (kUnroll - 1) * kThreads < part.end; k += kUnroll * kThreads) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) raw[i] = part.load(k + i * kThreads);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) take(raw[i], k + i * kThreads);
  }
  for (; k < part.end; k += kThreads) take(part.load(k), k);

  // the part's: largest logit, sum of exponentials under it, and of those times the
  // exponents (in powers of two)
  float high = block_reduce(most, s.red[0], [](float x, float y) { return fmaxf(x, y); });
  float z = 0.f, u = 0.f;
  const bool plain = high >= Bounds<T>::kLow && high <= kHigh;  // of the CTA
  if (plain) {
    if (most > Bounds<T>::kLowest) {
      const float d = (c - high) * kLog2e, f = exp2_fast(d);
      const float own = sum.x + sum.y;
      if (f > 0.f) {
        z = own * f;
        u = (mean.x + mean.y + own * d) * f;
      }
    }
  } else {
    float top = -INFINITY;
    for (int j = part.first + int(threadIdx.x); j < part.end; j += kThreads)
      part.each(j, [&](float v, int) { top = fmaxf(top, v); });
    __syncthreads();
    high = block_reduce(top, s.red[0], [](float x, float y) { return fmaxf(x, y); });
    for (int j = part.first + int(threadIdx.x); j < part.end; j += kThreads)
      part.each(j, [&](float v, int) {
        if (!(v > -INFINITY)) return;
        const float d = v == high ? 0.f : (v - high) * kLog2e, e = exp2f(d);
        z += e;
        if (e > 0.f) u += e * d;
      });
  }
  z = block_reduce(z, s.red[1], [](float x, float y) { return x + y; });
  u = block_reduce(u, s.red[2], [](float x, float y) { return x + y; });
  if (a.top && !(plain && pick<T>(part, a.top, most, at, s)))
    pick_slowly<T>(part, a.top, s);

  if (ranks > 1) {
    // to the first CTA of the cluster
    ptx::cluster_wait();  // it has started
    if (int(threadIdx.x) < a.top)
      st_cluster_u64(ptx::map_shared_rank(ptx::smem_u32(&s.all[rank][threadIdx.x]), 0u),
                     s.best[threadIdx.x]);
    if (threadIdx.x < 3)
      ptx::st_cluster_f32(ptx::map_shared_rank(ptx::smem_u32(&s.sums[rank][threadIdx.x]), 0u),
                          threadIdx.x == 0 ? high : threadIdx.x == 1 ? z : u);
    ptx::cluster_sync();
    if (rank) return;
    high = s.sums[0][0];
    for (int r = 1; r < ranks; ++r) high = fmaxf(high, s.sums[r][0]);
    z = u = 0.f;
    for (int r = 0; r < ranks; ++r) {
      const float h = s.sums[r][0];
      const float d = h == high ? 0.f : (h - high) * kLog2e, f = exp2f(d);
      if (f > 0.f) {
        z += s.sums[r][1] * f;
        u += (s.sums[r][2] + s.sums[r][1] * d) * f;
      }
    }
    // a logit's place among all lists: the number of better ones in each
    if (int(threadIdx.x) < a.top) s.best[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < ranks * a.top; i += kThreads) {
      const int own = i / a.top, j = i % a.top;
      const u64 p = s.all[own][j];
      int better = j;
      for (int r = 0; r < ranks; ++r)
        if (r != own) better += larger_in(s.all[r], a.top, p);
      if (p && better < a.top) s.best[better] = p;
    }
    __syncthreads();
  }
  // (the largest logit's own share makes z at least 1, and no term of u is above 0: what
  // rounding takes from there would make a log probability positive, an entropy negative)
  z = fmaxf(z, 1.f);
  u = fminf(u, 0.f);
  const float log_z = logf(z);
  auto logprob = [&](float v) {
    if (!(v > -INFINITY)) return -INFINITY;
    return (v == high ? 0.f : v - high) - log_z;
  };
  if (threadIdx.x == kThreads - 1) {
    const int t = a.tokens[m];
    a.logprobs[m] = t >= 0 && t < a.V ? logprob(widen(part.row[t])) : -INFINITY;
    a.entropy[m] = high > -INFINITY ? log_z - u / z * kLn2 : 0.f;
  }
  if (int(threadIdx.x) < a.top) {
    const u64 p = s.best[threadIdx.x];
    a.top_tokens[m * a.top + threadIdx.x] = p ? int32_t(~uint32_t(p)) : -1;
    a.top_logprobs[m * a.top + threadIdx.x] = logprob(value_of(uint32_t(p >> 32)));
  }
}

template <typename T>
void launch_t(const Args& a, int ranks, unsigned flags, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.M * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (ranks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(ranks);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (flags & QLIN_OVERLAP_PREVIOUS) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a, ranks);
}

template <typename T>
void dispatch(const Args& a, unsigned flags, cudaStream_t st) {
  // As many CTAs to a row as leave each thread 16 logits and an SM three CTAs.  (128256
  // logits in 16 bits, us, with two, three and four: 64 rows 12.9, 12.9 and 14.2, 100 rows
  // 17.1, 15.1 and 15.1, 150 rows 17.9, 17.9 and 23.5, 200 rows 23.9, 19.8 and 19.8.)
  const int64_t sms = sm_count();
  int ranks = 1;
  while (ranks < kMaxCluster && a.M * ranks * 2 <= 3 * sms && a.V / (ranks * 2) >= 16 * kThreads)
    ranks *= 2;
  launch_t<T>(a, ranks, flags, st);
}

}  // namespace

qlin_status launch_token_logprobs(const void* logits, int64_t stride, const int32_t* tokens,
                                  float* logprobs, float* entropy, int top, int32_t* top_tokens,
                                  float* top_logprobs, int64_t M, int64_t V, qlin_dtype ldtype,
                                  unsigned flags, cudaStream_t st) {
  const Args a = {logits, stride, tokens, logprobs, entropy, top, top_tokens, top_logprobs, M,
                  int(V)};
  if (ldtype == QLIN_F32)
    dispatch<float>(a, flags, st);
  else if (ldtype == QLIN_F16)
    dispatch<__half>(a, flags, st);
  else
    dispatch<__nv_bfloat16>(a, flags, st);
  return check_launch("qlin_token_logprobs");
}

}  // namespace qlin
