// Sampling a token per row of logits with temperature, top-k, top-p and min-p,
// from a given uniform number (qlin.h has the definition).
//
// A cluster of CTAs shares a row: each keeps its part of the row in shared
// memory, so the logits are read from memory once, and everything after works
// on the parts and exchanges a few words through distributed shared memory.
//
// What top-k and top-p keep is a beginning of the row's order (larger logits
// first, equal ones by index), so it is described by its last element.  A
// histogram over 2048 bins of equal width below the largest logit, of counts
// (top-k) or weights (top-p), tells the bin in which the sum from the top passes
// the bound.  The few elements of that bin go to one CTA, which sorts them and
// finds the last one kept; if they and all above them are few, for top-k and
// top-p at once.  Where they are many (equal logits, or a temperature that sets
// all of them apart or none), the element's logit is found digit by digit of its
// order-preserving bit pattern, by three more histograms.  (Histograms over the
// first digit in place of equal widths took 155 us for 96 rows of 128256: 40 bins
// held everything, and the atomics on them queued.)
//
// Weights are whole numbers of 2^-36, summed in limbs of 18 or 12 bits: the sums
// are exact, and the order of the atomic additions does not show.

#include <cmath>

#include "device_common.cuh"
#include "qlin_internal.h"
#include "sm100_ptx.cuh"

namespace qlin {

__device__ unsigned int g_sample_status = 0;  // 1: a bound that no bin passes

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 1024;  // elements that are sorted in one CTA
constexpr int kRankSort = 128;  // up to here by counting the larger ones
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

__device__ __forceinline__ void red_shared(uint32_t* p, uint32_t v) {
  asm volatile("red.shared.add.u32 [%0], %1;" ::"r"(ptx::smem_u32(p)), "r"(v));
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
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
  int limb;     // bits of the weights' limbs in a histogram
};

struct Shared {
  uint32_t hist[3][kBins];  // counts, or the weights' limbs
  u64 list[2 * kList];      // key << 32 | ~index, and room to sort
  float edges[kMaxCluster][8];  // weights down to the edges, of each rank
  uint32_t listed;
  int drawn;
  float drawn_prob;
  u64 warp_sum[kWarps], part_sum[kWarps];
  u64 exchange[2][kMaxCluster];
  u64 found[2][3];
};

// a/tau, rounded as the division rounds, for 1e-30 < tau < 1e30, |a| < 26 tau and
// quotients of 2^-30 or more (where a is subnormal, smaller ones can be off in their
// last bit; exp of them is 1).
// Markstein's (IBM J. Res. Dev. 34, 1990): with the reciprocal correctly rounded, a
// step that makes the quotient faithful and one that makes it correctly rounded,
// each on the exact remainder of a fused multiply-add.
__host__ __device__ inline float quotient(float a, float tau, float inverse) {
  float q = a * inverse;
  q = fmaf(fmaf(-q, tau, a), inverse, q);
  return fmaf(fmaf(-q, tau, a), inverse, q);
}

// exp((x - top)/tau), rounded as the division and expf round.  What weighs less
// than 2^-37 (quotients below -26) is 0, which also keeps infinities out of the
// quotient's steps.
struct Weigh {
  float top, tau, inverse, least;
  __device__ void set(float top_, float tau_) {
    top = top_;
    tau = tau_;
    inverse = __frcp_rn(tau);
    least = -26.0f * tau;
  }
  __device__ float operator()(float x) const {
    if (x == top) return 1.0f;
    const float a = x - top;
    if (!(a > least)) return 0.0f;
    if (tau == 1.0f) return expf(a);
    if (!(tau > 1e-30f && tau < 1e30f)) return expf(__fdiv_rn(a, tau));  // the steps' range
    return expf(quotient(a, tau, inverse));
  }
};
// rint(2^36 e), 0 <= e <= 1, as hi * 2^18 + lo with -2^17 <= lo <= 2^17.  Adding
// 2^23 rounds a smaller number to a whole one, to be read in the low bits; the
// remainder of the fused multiply-add is exact.  (The conversion to 64 bits has
// a quarter of an exponential's rate.)
struct Weight {
  int hi, lo;
  __device__ u64 sum() const { return (u64(uint32_t(hi)) << 18) + (long long)lo; }
};
__device__ __forceinline__ Weight split_weight(float e) {
  const float h = __fadd_rn(__fmul_rn(e, 0x1p18f), 0x1p23f);
  const float rest = fmaf(__fsub_rn(h, 0x1p23f), -0x1p18f, __fmul_rn(e, 0x1p36f));
  const float l = __fadd_rn(rest, 0x1.8p23f);
  return Weight{int(__float_as_uint(h) & 0x7fffffu), int(__float_as_uint(l)) - 0x4b400000};
}
__device__ __forceinline__ u64 weight_of(float e) { return split_weight(e).sum(); }

// What the loops over a part's elements go by: copied into registers by each.
template <typename T>
struct View {
  const T* x;   // the part, cleaned
  int n, base;  // its elements, and the first one's index
  Weigh weigh;
  // what is kept: up to this element of the order
  float last = -INFINITY;
  int last_index = 0x7fffffff;
  // bins of equal width for distances from the largest logit in [from, to)
  float from, to, scale;

  __device__ float at(int i) const { return logit<T>(x[i]); }
  __device__ bool in(int i, float v) const {
    return v > last || (v == last && base + i <= last_index);
  }
  // The bin of a logit: lower ones for larger logits, equal logits in one; -1
  // above the bins, kBins below.
  __device__ int bin_of(float v) const {
    const float d = v == weigh.top ? 0.f : weigh.top - v;
    if (d < from) return -1;
    if (d >= to && to < INFINITY) return kBins;
    const float b = (d - from) * scale;
    return b < kBins - 1 ? int(b) : kBins - 1;
  }
  // Bins for all: what lies below the 26th e-fold, and weighs nothing, goes to
  // the last one.
  __device__ void all_bins() {
    from = 0.f;
    to = INFINITY;
    scale = kBins / 26.0f * weigh.inverse;
  }
};

template <typename T>
struct Row {
  Shared& s;
  View<T> view;
  int rank, ranks;
  int limb;  // of every CTA of the cluster: they read each other's histograms
  float my_top;  // this thread's largest
  float u, min_p, below;
  int first_of_all;  // of the order
  int turn = 0;  // counts the exchanges: odd and even ones have buffers of their own

  __device__ Row(Shared& s_) : s(s_) {}

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

  // The first index whose cumulated count is above a target.  An element counts
  // 1 if it is kept and its logit is `to` (EQUAL; the target is `bound`), or its
  // weight if top-k, top-p and min-p keep it (the target is the draw's).  All
  // threads; the total and the count there come back too.  (The loops with an
  // exponential stand once in the code, and are not unrolled: else the kernel
  // outgrew the instruction cache and took three times as long.)
  template <bool EQUAL>
  __device__ __forceinline__ int find(float to, u64 bound, u64* total, u64* value) {
    const View<T>& r = view;
    const int n = r.n;
    const float least_p = min_p, low = below;
    const int always = first_of_all - r.base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = (n + kWarps * 32 - 1) / (kWarps * 32) * 32;  // of a warp
    const float least = EQUAL ? to : r.last;
    auto count_of = [&](int i, float v) -> u64 {
      if (!r.in(i, v)) return 0;
      if (EQUAL) return v == to;
      // (what is surely below min-p needs no exponential)
      if (v - r.weigh.top < low) return 0;
      const float e = r.weigh(v);
      return e >= least_p || i == always ? weight_of(e) : 0;
    };
    auto sum_of = [&](int i0, int i1) {
      u64 sum = 0;
#pragma unroll 1
      for (int i = i0 + lane; i < i1; i += 32) {
        const float v = r.at(i);
        if (v >= least) sum += count_of(i, v);
      }
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      return sum;
    };
    const int i0 = min(n, warp * share);
    const u64 sum = sum_of(i0, min(n, i0 + share));
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = sum;
    __syncthreads();
    u64 mine = 0;
    for (int i = 0; i < kWarps; ++i) mine += s.warp_sum[i];
    const u64* all = exchange(mine);
    u64 whole = 0, before = 0;
    for (int i = 0; i < ranks; ++i) {
      if (i == rank) before = whole;
      whole += all[i];
    }
    const u64 t = EQUAL ? bound : target(whole);
    u64* got = s.found[turn & 1];
    if (before <= t && t < before + mine) {  // this CTA has it (all its threads agree)
      int w = 0;                             // the warp whose share has it
      while (before + s.warp_sum[w] <= t) before += s.warp_sum[w++];
      // that share again, now in parts for all warps
      const int j1 = min(n, (w + 1) * share), part = (share / kWarps + 31) / 32 * 32;
      const int p0 = min(j1, w * share + warp * part), p1 = min(j1, p0 + part);
      const u64 sub = sum_of(p0, p1);
      if (lane == 0) s.part_sum[warp] = sub;
      __syncthreads();
      for (int i = 0; i < warp; ++i) before += s.part_sum[i];
      if (before <= t && t < before + sub) {
        for (int i = p0; i < p1; i += 32) {
          const u64 v = i + lane < p1 ? count_of(i + lane, r.at(i + lane)) : 0;
          u64 upto = v;
          for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
          }
          const unsigned past = __ballot_sync(0xffffffffu, before + upto > t);
          if (past) {
            const int l = __ffs(past) - 1;
            const u64 there = __shfl_sync(0xffffffffu, v, l);
            if (lane < ranks) {
              const uint32_t dst = ptx::map_shared_rank(ptx::smem_u32(got), lane);
              st_cluster_u64(dst, u64(r.base + i + l));
              st_cluster_u64(dst + 8, there);
            }
            break;
          }
          before += __shfl_sync(0xffffffffu, upto, 31);
        }
      }
    }
    ++turn;
    ptx::cluster_sync();
    *total = whole;
    *value = got[1];
    return int(got[0]);
  }

  // Sorts list[0 .. n) downward: each key to the place that the larger ones
  // leave it, or (bitonic) in the next power of two.
  __device__ void sort_list(int n) {
    if (n <= kRankSort) {
      u64* sorted = s.list + kList;
      if (int(threadIdx.x) < n) {
        const u64 mine = s.list[threadIdx.x];
        int larger = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) larger += s.list[i] > mine;
        sorted[larger] = mine;
      }
      __syncthreads();
      if (int(threadIdx.x) < n) s.list[threadIdx.x] = sorted[threadIdx.x];
      __syncthreads();
      return;
    }
    int size = 2;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int t = threadIdx.x; t < size / 2; t += kThreads) {
          const int i = 2 * t - (t & (j - 1));  // the lower of the pair i, i + j
          const u64 x = s.list[i], y = s.list[i + j];
          if ((x < y) == ((i & k) == 0)) {
            s.list[i] = y;
            s.list[i + j] = x;
          }
        }
        __syncthreads();
      }
  }

  // The inclusive sums of v over the threads, and the sum of all.
  __device__ u64 block_scan(u64 v, u64* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = 1; d < 32; d <<= 1) {
      const u64 w = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += w;
    }
    __syncthreads();
    if (lane == 31) s.warp_sum[warp] = v;
    __syncthreads();
    u64 sum = 0;
    for (int i = 0; i < kWarps; ++i) {
      if (i == warp) v += sum;
      sum += s.warp_sum[i];
    }
    *all = sum;
    return v;
  }

  // The draw, from a sorted list that holds all that top-k and top-p keep: its
  // first `limit` entries (at most kRankSort), two a thread.  One CTA.
  __device__ void draw_listed(int limit, const bool (&kept)[2], const float (&e)[2],
                              const u64 (&w)[2]) {
    u64* weight = s.list + kList;
    const int first = 2 * threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (first + i < limit)
        weight[first + i] = kept[i] && (first + i == 0 || e[i] >= min_p) ? w[i] : 0;
    __syncthreads();
    if (int(threadIdx.x) < limit) {
      // equal logits stand in the order of their indexes, the others do not: the
      // sum up to an index goes over all
      const uint32_t mine = ~uint32_t(s.list[threadIdx.x]);
      u64 total = 0, upto = 0;
#pragma unroll 4
      for (int i = 0; i < limit; ++i) {
        const u64 v = weight[i];
        total += v;
        upto += ~uint32_t(s.list[i]) <= mine ? v : 0;
      }
      const u64 t = target(total), own = weight[threadIdx.x];
      if (upto > t && upto - own <= t) {
        s.drawn = int(mine);
        s.drawn_prob = float(double(own) / double(total));
      }
    }
    __syncthreads();
  }

  // floor(u * total), within 0 .. total - 1.
  __device__ u64 target(u64 total) const {
    const double t = floor(double(u) * double(total));
    return t > 0.0 ? (t < double(total) ? u64(t) : total - 1) : 0;
  }

  // Where the sum over a histogram passes a bound.
  struct Cross {
    int bin;           // -1: nowhere
    u64 above, value;  // of the bins before it, and its own
  };
  enum What { kTops, kBands, kDigits };
  struct Digits {
    int bin;  // of the first histogram
    uint32_t prefix;
    int shift, bits;  // bits = 0: no digit so far, the prefix is empty
    bool begun;
  };

  // A histogram by count or by weight of the kept elements by their bins (kBands),
  // of each thread's largest element (kTops), or of those of a bin by a digit
  // (kDigits), and the first bin (0 first) in which `above` and the sum so far
  // pass a bound: reach k, or `mass`, or with mass < 0 the share p of all that is
  // counted.  What lies above the bins adds to `above`.
  __device__ __forceinline__ Cross histogram(What what, bool by_count, u64 above, u64 k, float p,
                                             double* mass, const Digits& digits) {
    const View<T>& r = view;
    const int n = r.n;
    const int arrays = by_count ? 1 : limb == 18 ? 2 : 3;
    const int count = what == kDigits ? 1 << digits.bits : kBins;
    for (int i = threadIdx.x; i < count; i += kThreads)
      for (int a = 0; a < arrays; ++a) s.hist[a][i] = 0;
    __syncthreads();
    u64 more = 0;
    if (what == kTops) {
      if (my_top > -INFINITY) red_shared(&s.hist[0][r.bin_of(my_top)], 1u);
    } else {
      const Digits dg = digits;
#pragma unroll 1
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float v = r.at(i);
        if (!r.in(i, v)) continue;
        int to = r.bin_of(v);
        if (what == kDigits) {
          const uint32_t q = key_of(v);
          if (to != dg.bin || (dg.begun && (q >> dg.shift >> dg.bits) != dg.prefix))
            continue;
          to = int(~(q >> dg.shift) & ((1u << dg.bits) - 1));  // larger ones first
        }
        if (to >= kBins) continue;
        if (by_count) {
          red_shared(&s.hist[0][to], 1u);
          continue;
        }
        const Weight w = split_weight(r.weigh(v));
        if (to < 0) {
          more += w.sum();
        } else if (limb == 18) {
          const uint32_t lo = w.lo & 0x3ffff, hi = w.hi + (w.lo >> 31);
          if (lo) red_shared(&s.hist[0][to], lo);
          if (hi) red_shared(&s.hist[1][to], hi);
        } else {
          const u64 all = w.sum();
          for (int a = 0; a < arrays; ++a)
            red_shared(&s.hist[a][to], uint32_t(all >> (12 * a)) & (a < 2 ? 0xfffu : ~0u));
        }
      }
    }
    ptx::cluster_sync();
    // each CTA adds up its share of the bins, rank 0 the first ones, each thread
    // a run of them
    const int share = count / ranks, run = max(1, share / kThreads);
    u64 v[4] = {0, 0, 0, 0}, mine = 0;
    const int first = rank * share + int(threadIdx.x) * run;
    if (int(threadIdx.x) * run < share) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < run) {
          for (int a = 0; a < arrays; ++a) {
            u64 sum = 0;
#pragma unroll 4
            for (int q = 0; q < ranks; ++q)
              sum += ld_cluster_u32(
                  ptx::map_shared_rank(ptx::smem_u32(&s.hist[a][first + i]), q));
            v[i] += sum << (limb * a);
          }
          mine += v[i];
        }
      }
    }
    u64 all, whole = 0;
    if (what == kBands && !by_count && r.from > 0.f) {
      block_scan(more, &all);
      const u64* firsts = exchange(all);
      for (int i = 0; i < ranks; ++i) above += firsts[i];
    }
    const u64 upto = block_scan(mine, &all);
    const u64* totals = exchange(all);
    u64 before = above + upto - mine;
    for (int i = 0; i < ranks; ++i) {
      if (i < rank) before += totals[i];
      whole += totals[i];
    }
    if (!by_count && *mass < 0.0) *mass = fmax(double(p) * double(whole), 0.5);
    if (by_count ? above + whole < k
                 : !(double(above) < *mass) || double(above + whole) < *mass)
      return Cross{-1, 0, 0};
    u64* got = s.found[turn & 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u64 after = before + v[i];
      const bool crosses = v[i] && (by_count ? before < k && after >= k
                                             : double(before) < *mass && !(double(after) < *mass));
      if (crosses) {
        for (int q = 0; q < ranks; ++q) {
          const uint32_t to = ptx::map_shared_rank(ptx::smem_u32(got), q);
          st_cluster_u64(to, u64(first + i));
          st_cluster_u64(to + 8, before);
          st_cluster_u64(to + 16, v[i]);
        }
      }
      before = after;
    }
    ++turn;
    ptx::cluster_sync();
    return Cross{int(got[0]), got[1], got[2]};
  }

  // The weight of the kept elements; the bins are set to a band of distances in
  // which the share p of it is passed.
  __device__ __forceinline__ u64 band(float p) {
    const View<T>& r = view;
    constexpr int kEdges = 8;
    constexpr float kEdge[kEdges] = {2.f, 4.f, 6.f, 8.f, 10.f, 12.f, 14.f, 17.f};  // e-folds
    float down[kEdges] = {};
    uint32_t hi = 0;
    int lo = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < r.n; i += kThreads) {
      const float v = r.at(i);
      if (!r.in(i, v)) continue;
      const float w = r.weigh(v);
      const float d = (r.weigh.top - v) * r.weigh.inverse;  // (NaN for infinities: in none)
      const Weight sw = split_weight(w);
      hi += sw.hi;
      lo += sw.lo;
#pragma unroll
      for (int e = 0; e < kEdges; ++e)
        if (d < kEdge[e]) down[e] += w;
    }
    const u64 sum = (u64(hi) << 18) + (long long)lo;  // (64 elements a thread at most)
    u64 all, whole = 0;
    block_scan(sum, &all);
    const u64* sums = exchange(all);
    for (int i = 0; i < ranks; ++i) whole += sums[i];
    // the edges' sums, over the CTA and then the cluster
#pragma unroll
    for (int e = 0; e < kEdges; ++e)
      for (int d = 16; d; d >>= 1) down[e] += __shfl_xor_sync(0xffffffffu, down[e], d);
    float* part = reinterpret_cast<float*>(s.hist[0]);  // [warp][edge]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < kEdges; ++e)
      if (lane == e) part[warp * kEdges + e] = down[e];
    __syncthreads();
    if (int(threadIdx.x) < kEdges) {
      float v = 0.f;
      for (int i = 0; i < kWarps; ++i) v += part[i * kEdges + threadIdx.x];
      for (int q = 0; q < ranks; ++q)
        ptx::st_cluster_f32(ptx::map_shared_rank(ptx::smem_u32(s.edges[rank] + threadIdx.x), q), v);
    }
    ptx::cluster_sync();
    const float bound = float(double(p) * double(whole) * 0x1p-36);
    float from = 0.f, end = 26.f * r.weigh.tau;
#pragma unroll
    for (int e = 0; e < kEdges; ++e) {
      float v = 0.f;
      for (int q = 0; q < ranks; ++q) v += s.edges[q][e];
      if (v < bound)
        from = kEdge[e] * r.weigh.tau;
      else
        end = fminf(end, kEdge[e] * r.weigh.tau);
    }
    if (from < end && end < INFINITY) {
      view.from = from;
      view.to = end;
      view.scale = kBins / (end - from);
    }
    return whole;
  }

  // The last element that a bound keeps: by count (the first k of the order) or
  // by weight (each whose predecessors weigh less than the share p of all), among
  // what was kept before.  By count it finds, where that costs nothing more, what
  // the share p keeps of the first k too, or draws the token.
  enum Found { kOne, kBoth, kDrawn };
  __device__ __forceinline__ Found cut(bool by_count, u64 k, float p) {
    double mass = -1.0;
    if (threadIdx.x == 0) s.listed = 0;
    view.all_bins();
    // For few, the threads' largest elements tell already: where k of them lie,
    // k elements do, and the list takes all down to that bin.  By weight, the sums
    // down to some distances, in registers, tell the band in which the bound lies,
    // and only its elements go through the histogram's atomics.
    What what = by_count && k <= u64(ranks * kThreads / 8) ? kTops : kBands;
    bool all_bins = by_count, list = true;
    if (!by_count) mass = fmax(double(p) * double(band(p)), 0.5);
    Digits digits = {0, 0, 21, 11, false};
    Cross c = {-1, 0, 0};
    while (true) {
      const Cross d = histogram(what, by_count, what == kDigits ? c.above : 0, k, p, &mass, digits);
      // (the sums are exact, so that over all bins, and over a bin's digits, one passes
      // the bound; if none did, the bound would be left out, not looked for again)
      if (d.bin < 0 && (what == kDigits || (what == kBands && all_bins))) {
        if (rank == 0 && threadIdx.x == 0) atomicOr(&g_sample_status, 1u);
        return kOne;
      }
      if (what == kDigits) {
        // too many for the list: digit by digit, of the elements of the bin
        digits.prefix =
            digits.prefix << digits.bits | (~uint32_t(d.bin) & ((1u << digits.bits) - 1));
        c.above = d.above;
        c.value = d.value;
        if (digits.shift == 0) break;
        digits.shift = digits.begun ? 0 : 10;
        digits.bits = digits.begun ? 10 : 11;
        digits.begun = true;
        continue;
      }
      c = d;
      if (c.bin < 0) {  // fewer threads have elements than k; or the band, which goes by
        what = kBands;  // rounded sums, was not the one
        all_bins = true;
        view.all_bins();
        continue;
      }
      // the list: those of the bin, or all down to it where they are few
      const bool whole = by_count && (what == kTops || c.above + c.value <= u64(kList));
      if (list && (!by_count || what == kTops || c.value <= u64(kList))) {
        list = false;
        const uint32_t to_count = ptx::map_shared_rank(ptx::smem_u32(&s.listed), 0);
        const uint32_t to_list = ptx::map_shared_rank(ptx::smem_u32(s.list), 0);
#pragma unroll 2
        for (int i = threadIdx.x; i < view.n; i += kThreads) {
          const float v = view.at(i);
          const int bin = view.bin_of(v);
          if (bin > c.bin || (bin < c.bin && !whole) || !view.in(i, v)) continue;
          uint32_t place;
          asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(place) : "r"(to_count));
          if (place < uint32_t(kList))
            st_cluster_u64(to_list + 8 * place, u64(key_of(v)) << 32 | uint32_t(~(view.base + i)));
        }
        ptx::cluster_sync();
        const bool both = whole && p < 1.f;
        u64* got = s.found[turn & 1];
        if (rank == 0) {
          const int count = int(s.listed);
          if (count > kList) {  // (by largest elements, or by weight: not counted before)
            if (int(threadIdx.x) < ranks)
              st_cluster_u64(ptx::map_shared_rank(ptx::smem_u32(got), threadIdx.x), 0);
          } else {
            sort_list(count);
            const u64 skipped = whole ? 0 : c.above;  // not in the list: elements, or weight
            const int limit = by_count ? int(k - skipped) : count;
            // two elements a thread, in order
            const int first = 2 * threadIdx.x;
            const bool by_mass = !by_count || both;
            const bool draws = whole && limit <= kRankSort;  // all that is kept is here, and few
            u64 w[2] = {0, 0}, all = 0, upto = 0;
            float e[2] = {0.f, 0.f};
            if (by_mass || draws) {
#pragma unroll 1
              for (int i = 0; i < 2; ++i)
                if (first + i < limit) {
                  const float x = view.weigh(of_key(uint32_t(s.list[first + i] >> 32)));
                  if (i == 0)
                    e[0] = x, w[0] = weight_of(x);
                  else
                    e[1] = x, w[1] = weight_of(x);
                }
              upto = block_scan(w[0] + w[1], &all);
            }
            if (both) mass = fmax(double(p) * double(all), 0.5);
            u64 before = upto - w[0] - w[1] + (by_count ? 0 : skipped);
            // the last kept: its predecessors weigh less, its successors' do not
            bool kept[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const u64 after = before + w[i];
              kept[i] = first + i < limit && !(by_mass && !(double(before) < mass));
              const bool next = first + i + 1 < limit && !(by_mass && !(double(after) < mass));
              if (kept[i] && !next)
                for (int q = 0; q < ranks; ++q)
                  st_cluster_u64(ptx::map_shared_rank(ptx::smem_u32(got), q), s.list[first + i]);
              before = after;
            }
            if (draws) draw_listed(limit, kept, e, w);
            if (int(threadIdx.x) < ranks)
              st_cluster_u64(ptx::map_shared_rank(ptx::smem_u32(got + 1), threadIdx.x), draws);
          }
        }
        ++turn;
        ptx::cluster_sync();
        if (got[0]) {  // (no element's entry is 0: its index's complement is not)
          view.last = of_key(uint32_t(got[0] >> 32));
          view.last_index = int(~uint32_t(got[0]));
          return got[1] ? kDrawn : both ? kBoth : kOne;
        }
      }
      if (what == kTops) {  // these took too many: count all elements
        what = kBands;
      } else {
        what = kDigits;
        digits.bin = c.bin;
      }
    }
    // of the elements with this logit the first `keep`
    const float to = of_key(digits.prefix);
    u64 keep, equal;
    if (by_count) {
      keep = k - c.above;
      equal = c.value;
    } else {
      const u64 w = weight_of(view.weigh(to));
      equal = c.value / w;
      keep = u64(fmax(1.0, ceil((mass - double(c.above)) / double(w))));
      while (keep > 1 && !(double(c.above + (keep - 1) * w) < mass)) --keep;
      while (keep < equal && double(c.above + keep * w) < mass) ++keep;
    }
    int index = to == view.last ? view.last_index : 0x7fffffff;
    if (keep < equal) {
      u64 total, ignored;
      index = find<true>(to, keep - 1, &total, &ignored);
    }
    view.last = to;
    view.last_index = index;
    return kOne;
  }
};

// The row of a cluster: of 512 rows those first whose bounds take longest, so that
// the last clusters to start are short ones.  (96 rows of 128256, a third of them
// with top-p alone: 128 us in the rows' own order, 110 in this.)
__device__ __forceinline__ int64_t row_of(const Params& a, int64_t y, int few, Shared& s) {
  const int64_t y0 = y / kThreads * kThreads;
  const int at = int(y - y0), rows = int(min(int64_t(kThreads), int64_t(gridDim.y) - y0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the largest or a few threads' maxima: 0; a draw among all: 1; a share of all: 2
  int cost = -1;
  if (int(threadIdx.x) < rows) {
    const int64_t m = y0 + threadIdx.x;
    const int k = a.top_k[m];
    cost = !(a.temperature[m] > 0.f) || (k > 0 && k <= few) ? 0 : a.top_p[m] < 1.f ? 2 : 1;
  }
  const int twos = __syncthreads_count(cost == 2), ones = __syncthreads_count(cost == 1);
  const int want = at < twos ? 2 : at < twos + ones ? 1 : 0;
  int skip = at - (want == 2 ? 0 : want == 1 ? twos : twos + ones);
  const unsigned mine = __ballot_sync(0xffffffffu, cost == want);
  if (lane == 0) s.warp_sum[warp] = __popc(mine);
  __syncthreads();
  for (int i = 0; i < warp; ++i) skip -= int(s.warp_sum[i]);
  if (cost == want && __popc(mine & ((1u << lane) - 1)) == skip) s.drawn = threadIdx.x;
  __syncthreads();
  return y0 + s.drawn;
}

// PER_SM: CTAs that an SM is to hold.
template <typename T, int PER_SM>
__global__ void __launch_bounds__(kThreads, PER_SM) sample_kernel(const Params a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  T* x = reinterpret_cast<T*>(raw + (sizeof(Shared) + 15) / 16 * 16);
  Row<T> row(s);
  row.view.x = x;
  row.rank = ptx::cluster_ctarank();
  row.ranks = gridDim.x;
  row.limb = a.limb;
  const int base = row.rank * a.part, n = max(0, min(a.part, a.V - base));
  row.view.base = base;
  row.view.n = n;
  // a peer's shared memory may be written to once the peer is known to have started;
  // the wait stands before the first exchange, behind the row's loads
  ptx::cluster_arrive_relaxed();
  grid_launch_dependents();
  grid_dependency_wait();
  // (one row for each cluster that fits: no order is better than another)
  const int64_t m = PER_SM == 1 ? blockIdx.y : row_of(a, blockIdx.y, row.ranks * kThreads / 8, s);
  const T* src = static_cast<const T*>(a.logits) + m * a.stride + base;

  // the part into shared memory, and the row's largest logit (the first such)
  u64 best = 0;
  float my_top = -INFINITY;
  int my_index = 0;
  auto look = [&](T v, int i) {
    const float c = clean(logit<T>(v));
    if (c > my_top) {  // (in a thread's order, equal ones come later)
      my_top = c;
      my_index = i;
    }
    return rounded<T>(c);
  };
  constexpr int kVec = 16 / sizeof(T);
  int done = 0;
  if (reinterpret_cast<uintptr_t>(src) % 16 == 0) {
    const int packs = n / kVec;
    done = packs * kVec;
#pragma unroll 4
    for (int i = threadIdx.x; i < packs; i += kThreads) {
      union {
        uint4 bits;
        T v[kVec];
      } u;
      u.bits = reinterpret_cast<const uint4*>(src)[i];
#pragma unroll
      for (int e = 0; e < kVec; ++e) u.v[e] = look(u.v[e], i * kVec + e);
      reinterpret_cast<uint4*>(x)[i] = u.bits;
    }
  }
#pragma unroll 4
  for (int i = done + threadIdx.x; i < n; i += kThreads) x[i] = look(src[i], i);
  // the row's first largest: a thread that saw nothing above -infinity may point
  // anywhere, which only shows in a row without a token
  best = u64(key_of(my_top)) << 32 | uint32_t(~(base + my_index));
  row.my_top = my_top;
  for (int d = 16; d; d >>= 1) {
    const u64 o = __shfl_xor_sync(0xffffffffu, best, d);
    best = o > best ? o : best;
  }
  if ((threadIdx.x & 31) == 0) s.warp_sum[threadIdx.x >> 5] = best;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) best = s.warp_sum[i] > best ? s.warp_sum[i] : best;
  ptx::cluster_wait();  // every CTA of the cluster has started
  const u64* all = row.exchange(best);
  for (int i = 0; i < row.ranks; ++i) best = all[i] > best ? all[i] : best;
  const int first = int(~uint32_t(best));
  row.view.weigh.set(of_key(uint32_t(best >> 32)), a.temperature[m]);

  int token;
  float prob;
  if (row.view.weigh.top == -INFINITY) {
    token = -1;
    prob = 0.f;
  } else if (!(row.view.weigh.tau > 0.f)) {
    token = first;
    prob = 1.f;
  } else {
    const int k = a.top_k[m];
    const float p = a.top_p[m] < 1.f ? fmaxf(a.top_p[m], 0.f) : 1.f, least = a.min_p[m];
    row.u = a.u[m];
    row.min_p = least;
    row.first_of_all = first;
    // (1e-3 is far more than the roundings of this bound and of the exponential)
    row.below = least > 0.f && least < 1.f ? row.view.weigh.tau * (logf(least) - 1e-3f) : -INFINITY;
    typename Row<T>::Found found = Row<T>::kOne;
#pragma unroll 1
    for (int by_count = 1; by_count >= 0; --by_count)  // top-k, then top-p
      if (found == Row<T>::kOne && (by_count ? k > 0 && k < a.V : p < 1.f))
        found = row.cut(by_count, k, p);
    if (found == Row<T>::kDrawn) {  // (by rank 0, which writes it)
      token = s.drawn;
      prob = s.drawn_prob;
    } else {
      u64 total, value;
      token = row.template find<false>(0.f, 0, &total, &value);
      prob = float(double(value) / double(total));
    }
  }
  if (row.rank == 0 && threadIdx.x == 0) {
    a.tokens[m] = token;
    if (a.probs) a.probs[m] = prob;
  }
  ptx::cluster_sync();  // no CTA leaves while a peer may still write to it
}

template <typename T, int PER_SM>
qlin_status launch_per_sm(const Params& a, int64_t M, int n, size_t bytes, unsigned flags,
                          cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  if (!allow_shared(reinterpret_cast<const void*>(sample_kernel<T, PER_SM>), 200 * 1024, &done))
    return check_launch("qlin_sample");
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
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
    cudaLaunchKernelEx(&cfg, sample_kernel<T, PER_SM>, p);
  }
  return check_launch("qlin_sample");
}

template <typename T>
qlin_status launch_t(Params a, int64_t M, unsigned flags, cudaStream_t st) {
  const int sms = sm_count();
  const SamplePlan p = sample_plan(M, a.V, sms);
  a.part = p.part;
  a.limb = p.limb;
  const size_t bytes = (sizeof(Shared) + 15) / 16 * 16 + size_t(p.part) * sizeof(T);
  // Where the clusters do not fill the SMs, all registers for one CTA (one row of
  // 128256: 19.4 us, 22.5 with room for two); else room for two (96 rows, in their
  // own order: 128 us, 194 with one).
  return M * p.ranks <= sms ? launch_per_sm<T, 1>(a, M, p.ranks, bytes, flags, st)
                            : launch_per_sm<T, 2>(a, M, p.ranks, bytes, flags, st);
}

}  // namespace

float sample_quotient(float a, float tau) { return quotient(a, tau, 1.0f / tau); }

SamplePlan sample_plan(int64_t M, int64_t V, int sms) {
  // CTAs that share a row: enough to fill the SMs twice, with 4096 elements or
  // more each; and below 16384 each, where weights take two atomics for three.  (Rows
  // of 128256, by this rule, by one that fills the SMs once, and by one that keeps to
  // one CTA an SM, us: 32 rows 70, 70, 99; 64 rows 89, 111, 169; 256 rows 281, 310, 310.)
  int64_t n = 1;
  while (n < kMaxCluster &&
         ((V + n - 1) / n + 7 >= 16384 || (M * n < 2 * sms && V > 4096 * 2 * n)))
    n *= 2;
  const int part = int(((V + n - 1) / n + 7) / 8 * 8);
  // Limbs whose sums over a part stay below 2^32.  It goes by the part's size, which
  // the row's CTAs have in common, not by how much of it the row fills.
  return SamplePlan{int(n), part, part < 16384 ? 18 : 12};
}

qlin_status launch_sample(const void* logits, int64_t logits_stride, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p,
                          const float* min_p, int32_t* tokens, float* probs, int64_t M,
                          int64_t V, qlin_dtype ldtype, unsigned flags, cudaStream_t st) {
  static_assert(kMaxVocab / kMaxCluster * 4 + sizeof(Shared) + 16 <= 200 * 1024, "a row fits");
  const Params a = {logits, logits_stride, u,      temperature, top_k, top_p,
                    min_p,  tokens,        probs,  int(V),      0,     0};
  switch (ldtype) {
    case QLIN_F16: return launch_t<__half>(a, M, flags, st);
    case QLIN_BF16: return launch_t<__nv_bfloat16>(a, M, flags, st);
    default: return launch_t<float>(a, M, flags, st);
  }
}

cudaError_t sample_take_device_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_sample_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_sample_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace qlin
