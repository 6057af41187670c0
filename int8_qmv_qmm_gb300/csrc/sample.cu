// Sampling a token per row of logits with temperature, top-k, top-p and min-p,
// from a given uniform number (qlin.h has the definition).
//
// A cluster of CTAs shares a row: each keeps its part of the row in shared
// memory, so the logits are read from memory once, and everything after works
// on the parts and exchanges a few words through distributed shared memory.
//
// What top-k and top-p keep is a beginning of the row's order (larger logits
// first, equal ones by index), so it is described by its last element.  That
// element's logit is found digit by digit (11, 11 and 10 bits of the logit's
// order-preserving bit pattern): a histogram of the counts (top-k) or weights
// (top-p) of the elements that share the digits found so far, and the first
// bin from the top in which the sum passes the bound.  Weights are whole
// numbers of 2^-36, summed in three 12-bit limbs: the sums are exact, and the
// order of the atomic additions does not show.

#include "device_common.cuh"
#include "qlin_internal.h"
#include "sm100_ptx.cuh"

namespace qlin {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxVocab = 262144;
using u64 = unsigned long long;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <typename T>
__device__ __forceinline__ float logit(T v);
template <>
__device__ __forceinline__ float logit<float>(float v) { return v; }
template <>
__device__ __forceinline__ float logit<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float logit<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// NaN counts as -infinity, and both zeros are one value.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.0f; }

// Larger floats have larger keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct Params {
  const void* logits;
  int64_t stride;
  const float *u, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  int32_t* tokens;
  float* probs;
  int V, part;  // elements of a row, and of a CTA's part
};

struct Shared {
  uint32_t hist[4][kBins];  // counts, or the weights' three limbs in 1 .. 3
  u64 warp_sum[kWarps];
  u64 exchange[2][kMaxCluster];
  u64 found[2][3];
  u64 picked;
};

__device__ __forceinline__ float exp_weight(float x, float top, float tau) {
  return x == top ? 1.0f : expf(__fdiv_rn(x - top, tau));
}
__device__ __forceinline__ u64 weight_of(float e) {
  return __float2ull_rn(e * 68719476736.0f);  // 2^36
}

template <typename T>
struct Row {
  Shared& s;
  const T* x;    // this CTA's part
  int n, base;   // its elements, and the first one's index
  int rank, ranks;
  float top, tau;
  int turn = 0;  // counts the exchanges: odd and even ones have buffers of their own

  __device__ Row(Shared& s_, const T* x_) : s(s_), x(x_) {}

  __device__ float at(int i) const { return clean(logit<T>(x[i])); }

  // Every CTA's v, in exchange[..][rank], after one cluster barrier.  A buffer
  // is written again two exchanges later, when the barrier in between has seen
  // every reader pass.
  __device__ const u64* exchange(u64 v) {
    u64* mine = s.exchange[turn & 1];
    ++turn;
    if (threadIdx.x < ranks)
      st_cluster_u64(ptx::map_shared_rank(ptx::smem_u32(mine + rank), threadIdx.x), v);
    ptx::cluster_sync();
    return mine;
  }

  // The sum over the CTA, in every thread.
  __device__ u64 block_sum(u64 v) {
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < kWarps; ++i) v += s.warp_sum[i];
    return v;
  }

  // The sum over the row.
  __device__ u64 row_sum(u64 v) {
    const u64* all = exchange(block_sum(v));
    u64 sum = 0;
    for (int i = 0; i < ranks; ++i) sum += all[i];
    return sum;
  }

  // The first index whose cumulated f is above bound(total); f(i, x) of the
  // part's element i.  All threads; total comes back too.
  template <class F, class B>
  __device__ int find(F f, B bound, u64* total, u64* value) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = (n + kWarps * 32 - 1) / (kWarps * 32) * 32;  // of a warp
    const int i0 = warp * share, i1 = min(n, i0 + share);
    u64 sum = 0;
    for (int i = i0 + lane; i < i1; i += 32) sum += f(i, at(i));
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = sum;
    __syncthreads();
    u64 mine = 0, before = 0;
    for (int i = 0; i < kWarps; ++i) {
      if (i == warp) before = mine;
      mine += s.warp_sum[i];
    }
    const u64* all = exchange(mine);
    u64 whole = 0;
    for (int i = 0; i < ranks; ++i) {
      if (i == rank) before += whole;
      whole += all[i];
    }
    const u64 t = bound(whole);
    u64* got = s.found[turn & 1];
    if (before <= t && t < before + sum) {  // this warp's share has it
      for (int i = i0; i < i1; i += 32) {
        const u64 v = i + lane < i1 ? f(i + lane, at(i + lane)) : 0;
        u64 upto = v;
        for (int d = 1; d < 32; d <<= 1) {
          const u64 w = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += w;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + upto > t);
        if (past) {
          const int l = __ffs(past) - 1;
          const u64 w = __shfl_sync(0xffffffffu, v, l);
          if (lane < ranks) {
            const uint32_t to = ptx::map_shared_rank(ptx::smem_u32(got), lane);
            st_cluster_u64(to, u64(base + i + l));
            st_cluster_u64(to + 8, w);
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    ++turn;
    ptx::cluster_sync();
    *total = whole;
    *value = got[1];
    return int(got[0]);
  }

  // The last element of the row's order that a bound keeps, among the elements
  // up to (key, index): by count (the first `k` of the order) or by weight
  // (each whose predecessors weigh less than `mass`).
  template <bool BY_COUNT>
  __device__ void cut(u64 k, double mass, uint32_t* key, int* index) {
    u64 above = 0, bin_value = 0;
    uint32_t prefix = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < kBins; i += kThreads)
        for (int a = BY_COUNT ? 0 : 1; a < (BY_COUNT ? 1 : 4); ++a) s.hist[a][i] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float v = at(i);
        const uint32_t q = key_of(v);
        if (pass && (q >> shift >> bits) != prefix) continue;
        if (q < *key || (q == *key && base + i > *index)) continue;
        const int bin = (q >> shift) & ((1 << bits) - 1);
        if (BY_COUNT) {
          atomicAdd(&s.hist[0][bin], 1u);
        } else {
          const u64 w = weight_of(exp_weight(v, top, tau));
          if (const uint32_t l = uint32_t(w & 0xfff)) atomicAdd(&s.hist[1][bin], l);
          if (const uint32_t l = uint32_t(w >> 12 & 0xfff)) atomicAdd(&s.hist[2][bin], l);
          if (const uint32_t l = uint32_t(w >> 24)) atomicAdd(&s.hist[3][bin], l);
        }
      }
      ptx::cluster_sync();
      // each CTA adds up its share of the bins, rank 0 the topmost, each thread
      // a run of them downward
      const int share = (1 << bits) / ranks, run = max(1, share / kThreads);
      u64 v[4] = {0, 0, 0, 0}, mine = 0;
      const int first = (1 << bits) - 1 - rank * share - int(threadIdx.x) * run;
      if (int(threadIdx.x) * run < share) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < run) {
            for (int p = 0; p < ranks; ++p)
              for (int a = BY_COUNT ? 0 : 1; a < (BY_COUNT ? 1 : 4); ++a)
                v[i] += u64(ld_cluster_u32(
                            ptx::map_shared_rank(ptx::smem_u32(&s.hist[a][first - i]), p)))
                        << (BY_COUNT ? 0 : 12 * (a - 1));
            mine += v[i];
          }
        }
      }
      u64 upto = mine;
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      for (int d = 1; d < 32; d <<= 1) {
        const u64 w = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += w;
      }
      __syncthreads();
      if (lane == 31) s.warp_sum[warp] = upto;
      __syncthreads();
      u64 all = 0, before = upto - mine;
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += s.warp_sum[i];
        all += s.warp_sum[i];
      }
      const u64* totals = exchange(all);
      before += above;
      for (int i = 0; i < rank; ++i) before += totals[i];
      u64* got = s.found[turn & 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (v[i]) {
          const u64 after = before + v[i];
          const bool crosses = BY_COUNT ? before < k && after >= k
                                        : double(before) < mass && !(double(after) < mass);
          if (crosses) {
            for (int p = 0; p < ranks; ++p) {
              const uint32_t to = ptx::map_shared_rank(ptx::smem_u32(got), p);
              st_cluster_u64(to, u64(first - i));
              st_cluster_u64(to + 8, before);
              st_cluster_u64(to + 16, v[i]);
            }
          }
          before = after;
        }
      }
      ++turn;
      ptx::cluster_sync();
      prefix = prefix << bits | uint32_t(got[0]);
      above = got[1];
      bin_value = got[2];
    }
    // all digits found: of the elements with this logit the first `keep`
    u64 keep, equal;
    if (BY_COUNT) {
      keep = k - above;
      equal = bin_value;
    } else {
      const u64 w = weight_of(exp_weight(of_key(prefix), top, tau));
      equal = bin_value / w;
      keep = u64(fmax(1.0, ceil((mass - double(above)) / double(w))));
      while (keep > 1 && !(double(above + (keep - 1) * w) < mass)) --keep;
      while (keep < equal && double(above + keep * w) < mass) ++keep;
    }
    if (keep < equal) {
      const uint32_t last_key = *key;
      const int last_index = *index;
      u64 total, value;
      *index = find(
          [&](int i, float v) -> u64 {
            return key_of(v) == prefix && (prefix > last_key || base + i <= last_index);
          },
          [&](u64) { return keep - 1; }, &total, &value);
    } else if (prefix != *key) {
      *index = 0x7fffffff;
    }
    *key = prefix;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const Params a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  T* x = reinterpret_cast<T*>(raw + (sizeof(Shared) + 15) / 16 * 16);
  Row<T> row(s, x);
  row.rank = ptx::cluster_ctarank();
  row.ranks = gridDim.x;
  const int64_t m = blockIdx.y;
  row.base = row.rank * a.part;
  row.n = max(0, min(a.part, a.V - row.base));
  grid_launch_dependents();
  grid_dependency_wait();
  const T* src = static_cast<const T*>(a.logits) + m * a.stride + row.base;

  // the part into shared memory, and the row's largest logit (the first such)
  u64 best = 0;
  for (int i = threadIdx.x; i < row.n; i += kThreads) {
    const T v = src[i];
    x[i] = v;
    const u64 k = u64(key_of(clean(logit<T>(v)))) << 32 | uint32_t(~(row.base + i));
    best = k > best ? k : best;
  }
  for (int d = 16; d; d >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, best, d);
    best = o > best ? o : best;
  }
  if ((threadIdx.x & 31) == 0) s.warp_sum[threadIdx.x >> 5] = best;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) best = s.warp_sum[i] > best ? s.warp_sum[i] : best;
  const u64* all = row.exchange(best);
  for (int i = 0; i < row.ranks; ++i) best = all[i] > best ? all[i] : best;
  const int first = int(~uint32_t(best));
  row.top = of_key(uint32_t(best >> 32));
  row.tau = a.temperature[m];

  int token;
  float prob;
  if (row.top == -INFINITY) {
    token = -1;
    prob = 0.f;
  } else if (!(row.tau > 0.f)) {
    token = first;
    prob = 1.f;
  } else {
    uint32_t key = 0;  // what is kept: up to this element of the order
    int index = 0x7fffffff;
    const int k = a.top_k[m];
    const float p = a.top_p[m], least = a.min_p[m];
    if (k > 0 && k < a.V) row.template cut<true>(k, 0.0, &key, &index);
    auto weight = [&](int i, float v) -> u64 {
      const uint32_t q = key_of(v);
      if (q < key || (q == key && row.base + i > index)) return 0;
      return weight_of(exp_weight(v, row.top, row.tau));
    };
    if (p < 1.f) {
      u64 mine = 0;
      for (int i = threadIdx.x; i < row.n; i += kThreads) mine += weight(i, row.at(i));
      const double mass = double(p) * double(row.row_sum(mine));
      row.template cut<false>(0, fmax(mass, 0.5), &key, &index);
    }
    auto kept = [&](int i, float v) -> u64 {
      const uint32_t q = key_of(v);
      if (q < key || (q == key && row.base + i > index)) return 0;
      const float e = exp_weight(v, row.top, row.tau);
      return e >= least || row.base + i == first ? weight_of(e) : 0;
    };
    const float u = a.u[m];
    u64 total, value;
    token = row.find(
        kept,
        [&](u64 sum) -> u64 {
          const double t = floor(double(u) * double(sum));
          return t > 0.0 ? (t < double(sum) ? u64(t) : sum - 1) : 0;
        },
        &total, &value);
    prob = float(double(value) / double(total));
  }
  if (row.rank == 0 && threadIdx.x == 0) {
    a.tokens[m] = token;
    if (a.probs) a.probs[m] = prob;
  }
  ptx::cluster_sync();  // no CTA leaves while a peer may still write to it
}

template <typename T>
qlin_status launch_t(Params a, int64_t M, unsigned flags, cudaStream_t st) {
  int n = 1;  // CTAs that share a row
  const int64_t header = (sizeof(Shared) + 15) / 16 * 16;
  auto bytes = [&](int r) { return header + ((a.V + r - 1) / r + 7) / 8 * 8 * int64_t(sizeof(T)); };
  while (n < kMaxCluster && bytes(n) > 200 * 1024) n *= 2;
  a.part = ((a.V + n - 1) / n + 7) / 8 * 8;
  if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           200 * 1024) != cudaSuccess)
    return check_launch("qlin_sample: cudaFuncSetAttribute");
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(bytes(n));
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 2 : 1;
  for (int64_t at = 0; at < M; at += 32768) {  // the grid's second axis ends at 65535
    Params p = a;
    p.logits = static_cast<const T*>(a.logits) + at * a.stride;
    p.u += at, p.temperature += at, p.top_k += at, p.top_p += at, p.min_p += at;
    p.tokens += at;
    if (p.probs) p.probs += at;
    cfg.gridDim = dim3(n, unsigned(M - at < 32768 ? M - at : 32768));
    cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
  }
  return check_launch("qlin_sample");
}

}  // namespace

qlin_status launch_sample(const void* logits, int64_t logits_stride, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p,
                          const float* min_p, int32_t* tokens, float* probs, int64_t M,
                          int64_t V, qlin_dtype ldtype, unsigned flags, cudaStream_t st) {
  static_assert(kMaxVocab / kMaxCluster * 4 + sizeof(Shared) + 16 <= 200 * 1024, "a row fits");
  const Params a = {logits, logits_stride, u,      temperature, top_k, top_p,
                    min_p,  tokens,        probs,  int(V),      0};
  switch (ldtype) {
    case QLIN_F16: return launch_t<__half>(a, M, flags, st);
    case QLIN_BF16: return launch_t<__nv_bfloat16>(a, M, flags, st);
    default: return launch_t<float>(a, M, flags, st);
  }
}

}  // namespace qlin
