// The experts' products where an expert has few rows: the packed weights stream past
// the tokens, and memory bounds it.
//
// mma.sync takes 16 weight rows as its rows and 8 of the expert's tokens as its
// columns, and works on the codes themselves: placed under the exponent of f16's 1024
// a code costs a byte permute (8 bits) or a mask (4 bits), and 1024 + q is exact.  Over
// a group of 64, with X = sum_k x_k and P = sum_k x_k (1024 + q_k),
//     sum_k x_k w_k = scale * P + (bias - 1024 * scale) * X,
// in float32: no weight is rounded.  (The 1024 costs P seven of its 24 bits at most, far
// below the output's rounding.)  Tokens in bfloat16 become f16 after a power of two for
// each group, which brings its largest element to 2^14: exact down to 2^-31 of that
// element, below which 2^-38 of it is lost at most.  (bfloat16 products on 8-bit codes
// would need two halves of each code: twice the products and masks.)
//
// A CTA, one on an SM, takes a run of items, each 16 rows for a tile of an expert's
// tokens.  Its 16 warps form teams that take items in turn, the warps of a team a share
// of K each.  The tile's tokens lie in shared memory in the order of the products'
// fragments, with the X of every group, for all items of the run that use them.  Each
// warp keeps a ring of stages in flight by its own cp.async, on through items and
// experts, so that the stream does not stop where a tile of tokens is fetched or sums
// are joined.
//
// 32 tokens of 8 of 64 experts of 2048 x 1024 at 8 bits, 135 MB, take 29 us, 4.6 TB/s; at
// 4 bits 31 us.  Neither memory (56% busy) nor the issue slots (50%, about 110 instructions
// for 16 rows of a group) are full: it waits for latencies between dependent instructions,
// fixed ones, shared memory's and the matrix products', which 16 warps an SM do not cover.
// One token of 8 experts of 2048 x 2048 at 4 bits, 19 MB, takes 11.7 us, of which 7 are
// launch, plan, tokens and the way of the first weights.

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "expert_plan.cuh"
#include "qlin_internal.h"
#include "sm100_ptx.cuh"

namespace qlin {

__device__ unsigned int g_expert_stream_status = 0;

namespace {

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_expert_stream_status, bit); }

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
// Warps of a team, which share an item's K.  (2, 4 and 8: 32 tokens' down in 33, 35 and 60
// us, one token's up in 13.2, 13.4 and 14.5.)
constexpr int kTeam = 2;
constexpr int kTeams = kWarps / kTeam;
// Tokens of a tile, a product's columns.  (With 16 and 32 of them: 36 and 36 us for 32;
// an expert that has more than 8 tokens finds its weights in L2.)
constexpr int kTokens = 8;
constexpr int kRows = 16;  // of an item
// Groups of a stage: 4, or 2 where that makes room for the tokens of a longer K.
constexpr int kManyGroups = 4, kFewGroups = 2;
template <int G>
constexpr int kRingBytes = 2048 * G;  // of a warp
constexpr int kScaleStride = kRows + 4;  // of a group's (scale, rest): spreads the banks
constexpr int kSumStride = kRows + 4;  // of a token's sums: spreads the banks
constexpr int kMaxExperts = 512;
constexpr int kCtasForJob = 4;
constexpr unsigned kAll = 0xffffffffu;

template <int BITS, int G>
constexpr int kStageBytes = G * kRows * 8 * BITS;
template <int BITS>
constexpr int kStages = 64 / (4 * BITS);  // 4 (4-bit) or 2

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d += a (16 x 16) b (16 x 8)
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A lane's 16 codes of a group (of rows g and g + 8) as the A operands of four products.
// Within a product's 16 elements of k the order is free, as long as the tokens' is the
// same: 8-bit codes pair up with their neighbours, 4-bit ones (a word at a time) as
// (0,4)(1,5) and (2,6)(3,7).
__device__ __forceinline__ void codes8(const uint4& w, int row, uint32_t (&a)[4][4]) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    a[s][row] = __byte_perm(words[s], 0x64646464u, 0x4140u);
    a[s][row + 2] = __byte_perm(words[s], 0x64646464u, 0x4342u);
  }
}
__device__ __forceinline__ void codes4(const uint2& w, int row, uint32_t (&a)[4][4]) {
  const uint32_t words[2] = {w.x, w.y};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t v = words[s / 2] >> (8 * (s % 2));
    a[s][row] = (v & 0x000f000fu) | 0x64006400u;
    a[s][row + 2] = ((v >> 4) & 0x000f000fu) | 0x64006400u;
  }
}

// Eight neighbours (four words of two) in the order of the products' B operands.
template <int BITS>
__device__ __forceinline__ uint4 in_order(uint4 v) {
  if constexpr (BITS == 8) return v;
  constexpr uint32_t kLow = 0x5410u, kHigh = 0x7632u;  // both low halves, both high ones
  return make_uint4(__byte_perm(v.x, v.z, kLow), __byte_perm(v.x, v.z, kHigh),
                    __byte_perm(v.y, v.w, kLow), __byte_perm(v.y, v.w, kHigh));
}

template <typename AT>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  const typename Act<AT>::T2 p = *reinterpret_cast<const typename Act<AT>::T2*>(&w);
  return make_float2(Act<AT>::to_f32(p.x), Act<AT>::to_f32(p.y));
}

// Of a token's group: X, and what its products are to be multiplied by (1 for f16).
struct TokenGroup {
  float x, back;
};

// Turns a quarter (16 elements) of a token's group, as loaded, into f16; the four lanes
// of the group call together.
template <typename AT>
__device__ __forceinline__ TokenGroup token_quarter(uint4& v0, uint4& v1) {
  uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float sum = 0.f;
  uint32_t most = 0u;  // the bits of magnitudes order as they do
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = widen2<AT>(w[i]);
    sum += f.x + f.y;
    most = max(most, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    sum += __shfl_xor_sync(kAll, sum, d);
    most = max(most, __shfl_xor_sync(kAll, most, d));
  }
  if constexpr (std::is_same<AT, __half>::value) return TokenGroup{sum, 1.f};
  // exponents of the largest: 14 after the factor; not where that passes float32's (the
  // element is then below 2^-100, or not finite)
  const int e = int(most >> 23);
  const int up = e < 27 ? 127 + 14 + 100 : e == 255 ? 127 : 127 + 14 + 127 - e;
  const float factor = __uint_as_float(uint32_t(up) << 23);
  const float back = __uint_as_float(uint32_t(254 - up) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = widen2<AT>(w[i]);
    const __half2 h = __floats2half2_rn(f.x * factor, f.y * factor);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  v0 = make_uint4(w[0], w[1], w[2], w[3]);
  v1 = make_uint4(w[4], w[5], w[6], w[7]);
  return TokenGroup{sum, back};
}

template <int BITS, typename AT, int kGroups>
__global__ void __launch_bounds__(kThreads, 1) stream_kernel(const ExpertArgs a) {
  constexpr int kAhead = kStages<BITS> - 1;
  static_assert(kStages<BITS> * kStageBytes<BITS, kGroups> == kRingBytes<kGroups>, "");
  extern __shared__ __align__(128) uint8_t shared[];
  __shared__ Jobs<kMaxExperts> plan;
  const int (&first_job)[kMaxExperts + 1] = plan.first;
  __shared__ int order[kThreads];  // where that holds all of it
  __shared__ int pair_of[kTokens];  // of the tile's tokens (-1: none)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wk = warp % kTeam, team = warp / kTeam;
  const int g = lane >> 2, c = lane & 3;
  const int n_groups = int(a.K) / kGroup, N = int(a.N);
  // rings | scales [kWarps][kGroups][kScaleStride] | sums [kWarps][kTokens][kSumStride] |
  // X and factors [n_groups][kTokens] | tokens
  float2* scales = reinterpret_cast<float2*>(shared + kWarps * kRingBytes<kGroups>) +
                   warp * kGroups * kScaleStride;
  float* sums = reinterpret_cast<float*>(shared + kWarps * (kRingBytes<kGroups> + kGroups * kScaleStride * 8));
  TokenGroup* xsum = reinterpret_cast<TokenGroup*>(sums + kWarps * kTokens * kSumStride);
  uint4* xs = reinterpret_cast<uint4*>(xsum + n_groups * kTokens);
  const uint8_t* ring = shared + warp * kRingBytes<kGroups>;
  // where this lane's copies go (4-bit: two groups of a row are 64 bytes, chunk c of row g
  // at chunk c ^ 2 * (g / 2 % 2), so that the reads below meet no bank twice)
  const uint32_t ring_to =
      ptx::smem_u32(ring) + uint32_t(BITS == 8 ? lane * 16 : g * 64 + (c ^ (g & 2)) * 16);

  const int ctas = int(gridDim.x), cta = int(blockIdx.x);
  grid_launch_dependents();
  grid_dependency_wait();
  // (a small plan is fetched whole beside its offsets, not after them)
  const bool small = a.n_pairs <= kThreads;
  if (small && int(threadIdx.x) < a.n_pairs) order[threadIdx.x] = a.order[threadIdx.x];
  if (fill_jobs(a, kTokens, plan) && cta == 0) report(kStatusPlan);
  const int blocks = (N + kRows - 1) / kRows;
  // The CTA's run of items: an equal share of all; where there are CTAs enough for each
  // job, one of a single job, whose tokens are then all that it fetches.
  const int jobs = first_job[a.E];
  const int64_t items = int64_t(jobs) * blocks;
  int64_t item0, item1;
  if (items <= 0x7fffffff) {  // (64-bit divisions take a good part of a microsecond)
    const unsigned each = unsigned(items) / ctas, more = unsigned(items) % ctas;
    item0 = each * cta + min(unsigned(cta), more);
    item1 = item0 + each + (unsigned(cta) < more ? 1 : 0);
  } else {
    item0 = items * cta / ctas;
    item1 = items * (cta + 1) / ctas;
  }
  if (jobs > 0 && kCtasForJob * jobs <= ctas) {
    const int job = cta * jobs / ctas;
    const int first = (job * ctas + jobs - 1) / jobs;  // of the job's CTAs
    const int n = ((job + 1) * ctas + jobs - 1) / jobs - first;
    item0 = int64_t(job) * blocks + int64_t(blocks) * (cta - first) / n;
    item1 = int64_t(job) * blocks + int64_t(blocks) * (cta - first + 1) / n;
  }
  const int n_items = int(item1 - item0);
  if (n_items == 0) return;

  // this warp's groups, and the stages that every warp of a team takes for an item
  const int g0 = wk * n_groups / kTeam, g1 = (wk + 1) * n_groups / kTeam;
  const int per_item = ((n_groups + kTeam - 1) / kTeam + kGroups - 1) / kGroups;
  const int64_t row_bytes = a.K * BITS / 8;

  // The team's items: a tile of an expert's tokens (job) and a block of rows.
  struct Place {
    int job, block, stage, left;  // left: items to come, this one too
  };
  Place now;
  now.job = items <= 0x7fffffff ? int(unsigned(item0) / unsigned(blocks)) : int(item0 / blocks);
  const int first = now.job;
  now.block = int(item0 - int64_t(first) * blocks) + team;
  now.stage = 0;
  now.left = (n_items - team + kTeams - 1) / kTeams;
  auto settle = [&](Place& q) {
    while (q.block >= blocks) {
      q.block -= blocks;
      ++q.job;
    }
  };
  if (now.left > 0) settle(now);
  // Where the copies are, ahead of the products: this lane's chunk of rows g and g + 8,
  // and the scale and bias of its group (c) there.
  Place ahead = now;
  // the expert of a job: first_job[expert] <= job < first_job[expert + 1]
  auto expert_of = [&](int job) {
    int low = 0, high = a.E;
    while (high - low > 1) {
      const int mid = (low + high) / 2;
      if (first_job[mid] <= job)
        low = mid;
      else
        high = mid;
    }
    return low;
  };
  int expert = ahead.left > 0 ? expert_of(ahead.job) : 0;  // ahead's
  const uint8_t* from[2];
  const uint16_t *scale_from[2], *bias_from[2];
  auto at_item = [&] {
    while (first_job[expert + 1] <= ahead.job) ++expert;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // (past the end: the last row, whose sums are not stored)
      const int64_t row = int64_t(expert) * N + min(ahead.block * kRows + 8 * half + g, N - 1);
      from[half] = reinterpret_cast<const uint8_t*>(a.wq) + row * row_bytes + g0 * (8 * BITS) + c * 16;
      scale_from[half] = static_cast<const uint16_t*>(a.scales) + row * n_groups + g0 + c;
      bias_from[half] = static_cast<const uint16_t*>(a.biases) + row * n_groups + g0 + c;
    }
  };
  if (ahead.left > 0) at_item();
  // scales and biases of the stages on their way (as loaded: nothing may touch them, and
  // so wait for them, before their stage); 0 for a group past the warp's last, which then
  // adds nothing
  uint16_t coming[kAhead + 1][2][2];
  int slot_in = 0;  // of the ring
  auto fetch = [&] {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        coming[i][half][0] = coming[i + 1][half][0];
        coming[i][half][1] = coming[i + 1][half][1];
      }
    if (ahead.left > 0) {
      const int n = min(g1 - g0 - ahead.stage * kGroups, kGroups);  // groups
      const uint32_t to = ring_to + uint32_t(slot_in * kStageBytes<BITS, kGroups>);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if constexpr (BITS == 8) {
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
            if (i < n) copy16(to + uint32_t((i * 2 + half) * 512), from[half] + i * 64);
        } else {
#pragma unroll
          for (int i = 0; i < kGroups; i += 2)
            if (i + c / 2 < n) copy16(to + uint32_t((i + half) * 512), from[half] + i * 32);
        }
        coming[kAhead][half][0] = c < n ? *scale_from[half] : uint16_t(0);
        coming[kAhead][half][1] = c < n ? *bias_from[half] : uint16_t(0);
        from[half] += kGroups * 8 * BITS;
        scale_from[half] += kGroups;
        bias_from[half] += kGroups;
      }
      if (++ahead.stage == per_item) {
        ahead.stage = 0;
        if (--ahead.left > 0) {
          ahead.block += kTeams;
          settle(ahead);
          at_item();
        }
      }
    }
    copies_commit();
    if (++slot_in == kStages<BITS>) slot_in = 0;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch();

  float2 acc[2];
  int slot = 0;
  const int64_t past = item0 + n_items;
  for (int job = first; int64_t(job) * blocks < past; ++job) {
    // the job's tokens
    const int of = expert_of(job), t0 = (job - first_job[of]) * kTokens;
    int p = -1;
    if (threadIdx.x < kTokens && t0 + int(threadIdx.x) < plan.count[of]) {
      const int at = plan.row[of] + t0 + threadIdx.x;
      p = small ? order[at] : a.order[at];
      if (p < 0 || p >= a.n_pairs) {
        report(kStatusPlan);
        p = -1;
      }
    }
    __syncthreads();  // (every team is done with the last job's)
    if (threadIdx.x < kTokens) pair_of[threadIdx.x] = p;
    __syncthreads();
    for (int i = threadIdx.x; i < n_groups * 32; i += kThreads) {
      const int q = i & 3, tok = (i >> 2) & 7, gr = i >> 5;
      const int pair = pair_of[tok];
      uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
      if (pair >= 0) {
        const uint4* x = reinterpret_cast<const uint4*>(
            static_cast<const AT*>(a.x) + int64_t(pair / a.pairs_per_row) * a.x_stride +
            gr * kGroup + q * 16);
        v0 = x[0];
        v1 = x[1];
      }
      const TokenGroup tg = token_quarter<AT>(v0, v1);  // (i runs in whole warps)
      if (q == 0) xsum[gr * kTokens + tok] = tg;
      uint4* to = xs + gr * 64 + tok * 4 + q;
      to[0] = in_order<BITS>(v0);
      to[32] = in_order<BITS>(v1);
    }
    __syncthreads();
    while (now.left > 0 && now.job == job) {
      __syncwarp();  // every lane is done with the stage whose place is filled next
      fetch();
      if (now.stage == 0) acc[0] = acc[1] = make_float2(0.f, 0.f);
      // (scale, bias - 1024 * scale) of group c, for the warp
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float scale = Act<AT>::to_f32(*reinterpret_cast<const AT*>(&coming[0][half][0]));
        const float bias = Act<AT>::to_f32(*reinterpret_cast<const AT*>(&coming[0][half][1]));
        if (c < kGroups)
          scales[c * kScaleStride + 8 * half + g] = make_float2(scale, fmaf(-1024.f, scale, bias));
      }
      copies_wait<kAhead>();
      __syncwarp();
      const uint8_t* st = ring + slot * kStageBytes<BITS, kGroups>;
      if (++slot == kStages<BITS>) slot = 0;
      const int s0 = g0 + now.stage * kGroups;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        uint32_t code[4][4];
        float2 sz[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if constexpr (BITS == 8)
            codes8(*reinterpret_cast<const uint4*>(st + (i * 2 + half) * 512 + lane * 16), half,
                   code);
          else
            codes4(*reinterpret_cast<const uint2*>(
                       st + (i / 2 * 2 + half) * 512 + g * 64 +
                       ((i % 2 * 2 + c / 2) ^ (g & 2)) * 16 + c % 2 * 8),
                   half, code);
          sz[half] = scales[i * kScaleStride + 8 * half + g];
        }
        // (past the warp's last group its tokens again: what is finite times 0)
        const int gr = max(min(s0 + i, g1 - 1), 0);
        const uint4 b0 = xs[gr * 64 + lane], b1 = xs[gr * 64 + 32 + lane];
        // of tokens 2c and 2c + 1
        const float4 tg = *reinterpret_cast<const float4*>(xsum + gr * kTokens + 2 * c);
        float p0[4] = {0.f, 0.f, 0.f, 0.f}, p1[4] = {0.f, 0.f, 0.f, 0.f};
        mma(p0, code[0], b0.x, b0.y);
        mma(p1, code[2], b1.x, b1.y);
        mma(p0, code[1], b0.z, b0.w);
        mma(p1, code[3], b1.z, b1.w);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float2 v = __fadd2_rn(make_float2(p0[2 * half], p0[2 * half + 1]),
                                make_float2(p1[2 * half], p1[2 * half + 1]));
          if constexpr (!std::is_same<AT, __half>::value)
            v = __fmul2_rn(v, make_float2(tg.y, tg.w));
          acc[half] = __ffma2_rn(make_float2(sz[half].y, sz[half].y), make_float2(tg.x, tg.z),
                                 acc[half]);
          acc[half] = __ffma2_rn(make_float2(sz[half].x, sz[half].x), v, acc[half]);
        }
      }
      const int block = now.block;
      if (++now.stage < per_item) continue;
      now.stage = 0;
      if (--now.left > 0) {
        now.block += kTeams;
        settle(now);
      }
      // the item's sums: rows g, g + 8 and tokens 2c, 2c + 1 from every warp of the team
      float* mine = sums + team * kTeam * kTokens * kSumStride;
      auto team_sync = [&] {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(kTeam * 32) : "memory");
      };
      team_sync();  // the team has read the last item's
      float* part = mine + wk * kTokens * kSumStride;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        part[2 * c * kSumStride + 8 * half + g] = acc[half].x;
        part[(2 * c + 1) * kSumStride + 8 * half + g] = acc[half].y;
      }
      team_sync();
      for (int i = wk * 32 + lane; i < kTokens * kRows; i += kTeam * 32) {
        const int tok = i / kRows, row = block * kRows + i % kRows;
        const int pair = pair_of[tok];
        if (pair < 0 || row >= N) continue;
        const float* sum = mine + tok * kSumStride + i % kRows;
        float v = sum[0];
#pragma unroll
        for (int k = 1; k < kTeam; ++k) v += sum[k * kTokens * kSumStride];
        if (a.y_f32)
          static_cast<float*>(a.y)[int64_t(pair) * N + row] = v;
        else
          static_cast<AT*>(a.y)[int64_t(pair) * N + row] = Act<AT>::from_f32_rn(v);
      }
    }
  }
  copies_wait<0>();
}

size_t shared_bytes(int64_t K, int groups) {
  return size_t(kWarps) * (2048 * groups + groups * kScaleStride * 8 + kTokens * kSumStride * 4) +
         size_t(K / kGroup) * kTokens * (sizeof(TokenGroup) + kGroup * 2);
}

constexpr size_t kMostShared = 227 * 1024 - 8704;  // beside the plan

template <int BITS, typename AT, int G>
qlin_status launch_g(const ExpertArgs& a, unsigned flags, cudaStream_t st) {
  auto kern = stream_kernel<BITS, AT, G>;
  static std::atomic<unsigned long long> done{0};
  if (!allow_shared(reinterpret_cast<const void*>(kern), int(kMostShared), &done))
    return check_launch("qlin_expert_linear: shared memory");
  // tiles of tokens: at most one more than full ones for each expert that has any
  const int64_t used = std::min<int64_t>(a.E, a.n_pairs);
  const int64_t jobs = a.n_pairs / kTokens + used;
  const int64_t items = jobs * ((a.N + kRows - 1) / kRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(items, sm_count())));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared_bytes(a.K, G);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kern, a);
  return check_launch("qlin_expert_linear");
}

template <int BITS, typename AT>
qlin_status launch_t(const ExpertArgs& a, unsigned flags, cudaStream_t st) {
  return shared_bytes(a.K, kManyGroups) <= kMostShared
             ? launch_g<BITS, AT, kManyGroups>(a, flags, st)
             : launch_g<BITS, AT, kFewGroups>(a, flags, st);
}

}  // namespace

bool expert_stream_fits(int64_t K) { return shared_bytes(K, kFewGroups) <= kMostShared; }

qlin_status launch_expert_stream(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st) {
  if (dtype == QLIN_F16)
    return bits == 4 ? launch_t<4, __half>(a, flags, st) : launch_t<8, __half>(a, flags, st);
  return bits == 4 ? launch_t<4, __nv_bfloat16>(a, flags, st)
                   : launch_t<8, __nv_bfloat16>(a, flags, st);
}

cudaError_t expert_stream_take_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_expert_stream_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_expert_stream_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace qlin
