// The experts' products where an expert has few rows: the packed weights stream past
// the tokens, and memory bounds it.
//
// mma.sync takes 16 weight rows as its rows and 8 of the expert's tokens as its
// columns, and works on the codes themselves: placed under the exponent of a 16-bit
// unit (f16 1024 + q, bfloat16 128 + q; 8-bit codes in bfloat16 by halves of 4 bits,
// 128 + low and 2048 + 16 high) a code costs one byte permute or mask, and is exact.
// Over a group of 64, with X = sum_k x_k and P = sum_k x_k (unit + q_k),
//     sum_k x_k w_k = scale * P + (bias - unit * scale) * X,
// in float32: no weight is rounded.  (The unit costs P seven of its 24 bits at most,
// far below the output's rounding.)
//
// A CTA takes a run of (expert, tile of tokens, 16 or more rows) items; its eight warps
// share an item's K and, where K is short, 16 rows each of several.  The tile's tokens
// lie in shared memory in the order of the products' fragments, with the X of every
// group, for all items of the run that use them.  Each warp keeps a ring of stages of
// four groups in flight by its own cp.async, on through items and experts, so that the
// stream does not stop where a tile of tokens is fetched or sums are joined.

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

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kGroups = 4;            // of a stage
constexpr int kRows = 16;             // weight rows of a warp
constexpr int kRingBytes = 8 * 1024;  // of a warp
constexpr int kMaxExperts = 512;
constexpr unsigned kAll = 0xffffffffu;

template <int BITS>
struct Ring {
  static constexpr int kStageBytes = kGroups * kRows * 8 * BITS;
  static constexpr int kStages = kRingBytes / kStageBytes;  // 4 (4-bit) or 2
};

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
template <typename AT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<AT, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What a code is placed in, and how a lane's 16 codes of a group become the A operands
// of four products (two of each for 8 bits in bfloat16), two pairs of codes to each.
// kOrder: how tokens' elements pair up to match: 0 neighbours, 1 (0,2)(1,3) of four,
// 2 (0,4)(1,5)(2,6)(3,7) of eight.
template <int BITS, typename AT>
struct Codes;

template <>
struct Codes<8, __half> {
  static constexpr float kUnit = 1024.f;
  static constexpr int kOrder = 0, kParts = 1;
  static __device__ __forceinline__ void pairs(const uint32_t (&w)[4], int s, int,
                                               uint32_t& p0, uint32_t& p1) {
    p0 = __byte_perm(w[s], 0x64646464u, 0x4140u);
    p1 = __byte_perm(w[s], 0x64646464u, 0x4342u);
  }
};
template <>
struct Codes<8, __nv_bfloat16> {
  static constexpr float kUnit = 128.f + 2048.f;
  static constexpr int kOrder = 1, kParts = 2;
  static __device__ __forceinline__ void pairs(const uint32_t (&w)[4], int s, int part,
                                               uint32_t& p0, uint32_t& p1) {
    const uint32_t unit = part ? 0x45004500u : 0x43004300u;
    p0 = ((w[s] >> (4 * part)) & 0x000f000fu) | unit;
    p1 = ((w[s] >> (4 * part + 8)) & 0x000f000fu) | unit;
  }
};
template <typename AT>
struct Codes<4, AT> {
  static constexpr float kUnit = std::is_same<AT, __half>::value ? 1024.f : 128.f;
  static constexpr int kOrder = 2, kParts = 1;
  static __device__ __forceinline__ void pairs(const uint32_t (&w)[2], int s, int,
                                               uint32_t& p0, uint32_t& p1) {
    p0 = ((w[s / 2] >> (8 * (s % 2))) & 0x000f000fu) | Act<AT>::kMagic2;
    p1 = ((w[s / 2] >> (8 * (s % 2) + 4)) & 0x000f000fu) | Act<AT>::kMagic2;
  }
};

// Eight neighbours (four words of two) in the order of the products' B operands.
template <int ORDER>
__device__ __forceinline__ uint4 in_order(uint4 v) {
  if constexpr (ORDER == 0) return v;
  constexpr uint32_t kLow = 0x5410u, kHigh = 0x7632u;  // both low halves, both high ones
  if constexpr (ORDER == 1)
    return make_uint4(__byte_perm(v.x, v.y, kLow), __byte_perm(v.x, v.y, kHigh),
                      __byte_perm(v.z, v.w, kLow), __byte_perm(v.z, v.w, kHigh));
  return make_uint4(__byte_perm(v.x, v.z, kLow), __byte_perm(v.x, v.z, kHigh),
                    __byte_perm(v.y, v.w, kLow), __byte_perm(v.y, v.w, kHigh));
}

template <typename AT>
__device__ __forceinline__ float sum8(uint4 v) {
  using T2 = typename Act<AT>::T2;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T2 p = *reinterpret_cast<const T2*>(&w[i]);
    s += Act<AT>::to_f32(p.x) + Act<AT>::to_f32(p.y);
  }
  return s;
}

// NT: tiles of 8 tokens; WK: warps that share a row's K (8 / WK blocks of 16 rows an
// item).
template <int BITS, typename AT, int NT, int WK>
__global__ void __launch_bounds__(kThreads, NT == 4 ? 1 : 2) stream_kernel(const ExpertArgs a) {
  using C = Codes<BITS, AT>;
  using R = Ring<BITS>;
  constexpr int kTokens = 8 * NT, WN = kWarps / WK, kItemRows = kRows * WN;
  constexpr int kSumStride = kItemRows + 4;  // (of a token: spreads the banks)
  constexpr int kLaneBytes = 2 * BITS;       // of a lane's 16 codes of a group
  extern __shared__ __align__(128) uint8_t shared[];
  __shared__ int first_job[kMaxExperts + 1];  // the tiles of the experts before each
  __shared__ int pair_of[2][kTokens];         // of the tile's tokens (-1: none)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wk = warp % WK, wn = warp / WK;
  const int g = lane >> 2, c = lane & 3;
  const int n_groups = int(a.K) / kGroup;
  // rings | sums [2][WK][kTokens][kSumStride] | X [n_groups][kTokens] | tokens
  float* sums = reinterpret_cast<float*>(shared + kWarps * kRingBytes);
  float* xsum = sums + 2 * WK * kTokens * kSumStride;
  uint4* xs = reinterpret_cast<uint4*>(xsum + n_groups * kTokens);
  const uint8_t* ring = shared + warp * kRingBytes;
  const uint32_t ring_u32 = ptx::smem_u32(ring);

  grid_launch_dependents();
  grid_dependency_wait();
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const ExpertRows r = expert_rows(a, e);
    if (r.bad && blockIdx.x == 0) report(kStatusPlan);
    first_job[e + 1] = (r.n + kTokens - 1) / kTokens;
  }
  if (threadIdx.x == 0) first_job[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int e0 = 1; e0 <= a.E; e0 += 32) {
      int v = e0 + lane <= a.E ? first_job[e0 + lane] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, v, d);
        if (lane >= d) v += o;
      }
      if (e0 + lane <= a.E) first_job[e0 + lane] = before + v;
      before += __shfl_sync(kAll, v, 31);
    }
  }
  __syncthreads();
  const int blocks = int((a.N + kItemRows - 1) / kItemRows);
  const int64_t items = int64_t(first_job[a.E]) * blocks;
  const int64_t item0 = items * blockIdx.x / gridDim.x;
  const int n_items = int(items * (blockIdx.x + 1) / gridDim.x - item0);
  if (n_items == 0) return;

  // this warp's groups, and the stages that every warp takes for an item
  const int g0 = wk * n_groups / WK, g1 = (wk + 1) * n_groups / WK;
  const int per_item = ((n_groups + WK - 1) / WK + kGroups - 1) / kGroups;

  // where a stage is: an item and a stage of it
  struct Cursor {
    int job, expert, block, stage, left;  // left: stages to the end of the run
  };
  auto at_expert = [&](Cursor& q) {
    while (first_job[q.expert + 1] <= q.job) ++q.expert;
  };
  auto next = [&](Cursor& q) {
    --q.left;
    if (++q.stage < per_item) return;
    q.stage = 0;
    if (++q.block < blocks) return;
    q.block = 0;
    ++q.job;
    if (q.left > 0) at_expert(q);
  };
  Cursor now;
  now.job = int(item0 / blocks);
  now.block = int(item0 % blocks);
  now.expert = now.stage = 0;
  now.left = n_items * per_item;
  at_expert(now);
  Cursor ahead = now;

  const int row_bytes = int(a.K) * BITS / 8;
  // row r of the item (past the end: the last one, whose sums are not stored)
  auto row_of = [&](const Cursor& q, int half) {
    const int64_t n = int64_t(q.block) * kItemRows + wn * kRows + 8 * half + g;
    return int64_t(q.expert) * a.N + min(n, a.N - 1);
  };
  int slot_in = 0;  // of the ring
  auto fetch = [&] {
    if (ahead.left > 0) {
      const int s0 = g0 + ahead.stage * kGroups, n = min(kGroups, g1 - s0);
      const uint32_t to = ring_u32 + uint32_t(slot_in * R::kStageBytes);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint8_t* from = reinterpret_cast<const uint8_t*>(a.wq) +
                              row_of(ahead, half) * row_bytes + s0 * (8 * BITS) + c * 16;
        if constexpr (BITS == 8) {
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
            if (i < n) copy16(to + uint32_t(((i * 2 + half) * 32 + lane) * 16), from + i * 64);
        } else {
          // two groups of a row are 64 bytes: chunk c of row g at chunk c ^ 2 * (g / 2 % 2)
#pragma unroll
          for (int i = 0; i < kGroups; i += 2)
            if (i + c / 2 < n)
              copy16(to + uint32_t(((i / 2 * 2 + half) * 8 + g) * 64 + (c ^ (g & 2)) * 16),
                     from + i * 32);
        }
      }
      next(ahead);
    }
    copies_commit();
    if (++slot_in == R::kStages) slot_in = 0;
  };
  // scale and bias (low and high half) of the stage's group c, rows g and g + 8
  uint32_t sb[2] = {0u, 0u};
  auto scales_of = [&](const Cursor& q) {
    const int gr = g0 + q.stage * kGroups + c;
    if (q.left > 0 && gr < g1) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t i = row_of(q, half) * n_groups + gr;
        sb[half] = uint32_t(static_cast<const uint16_t*>(a.scales)[i]) |
                   uint32_t(static_cast<const uint16_t*>(a.biases)[i]) << 16;
      }
    }
  };

#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) fetch();
  scales_of(now);

  float acc[NT][4];
  int slot = 0, sum_buf = 0, tile_buf = 0, tile = -1;
  while (now.left > 0) {
    __syncwarp();  // every lane is done with the stage whose place is filled next
    fetch();
    if (now.job != tile) {
      // the tokens of another tile (every warp is past the last item's products: its
      // barrier lies behind them)
      tile = now.job;
      tile_buf ^= 1;
      const ExpertRows r = expert_rows(a, now.expert);
      const int t0 = (now.job - first_job[now.expert]) * kTokens;
      if (threadIdx.x < kTokens) {
        int p = -1;
        if (t0 + int(threadIdx.x) < r.n) {
          p = a.order[r.first + t0 + threadIdx.x];
          if (p < 0 || p >= a.n_pairs) {
            report(kStatusPlan);
            p = -1;
          }
        }
        pair_of[tile_buf][threadIdx.x] = p;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < n_groups * kTokens * 4; i += kThreads) {
        const int q = i & 3, tok = (i >> 2) % kTokens, gr = (i >> 2) / kTokens;
        const int p = pair_of[tile_buf][tok];
        uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
        if (p >= 0) {
          const uint4* from = reinterpret_cast<const uint4*>(
              static_cast<const AT*>(a.x) + int64_t(p / a.pairs_per_row) * a.x_stride +
              gr * kGroup + q * 16);
          v0 = from[0];
          v1 = from[1];
        }
        float s = sum8<AT>(v0) + sum8<AT>(v1);
        s += __shfl_xor_sync(kAll, s, 1);  // (i runs in whole warps)
        s += __shfl_xor_sync(kAll, s, 2);
        if (q == 0) xsum[gr * kTokens + tok] = s;
        uint4* to = xs + ((gr * NT + tok / 8) * 2) * 32 + (tok % 8) * 4 + q;
        to[0] = in_order<C::kOrder>(v0);
        to[32] = in_order<C::kOrder>(v1);
      }
      __syncthreads();
    }
    if (now.stage == 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
    }
    const uint32_t sb_now[2] = {sb[0], sb[1]};
    const Cursor it = now;
    next(now);
    scales_of(now);
    copies_wait<R::kStages - 1>();
    if constexpr (BITS == 4) __syncwarp();
    const int s0 = g0 + it.stage * kGroups, n = min(kGroups, g1 - s0);
    const uint8_t* st = ring + slot * R::kStageBytes;
    if (++slot == R::kStages) slot = 0;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      if (i >= n) break;
      uint32_t w[2][kLaneBytes / 4];  // rows g and g + 8: 16 codes each
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if constexpr (BITS == 8) {
          const uint4 v = *reinterpret_cast<const uint4*>(st + ((i * 2 + half) * 32 + lane) * 16);
          w[half][0] = v.x, w[half][1] = v.y, w[half][2] = v.z, w[half][3] = v.w;
        } else {
          const int chunk = (i % 2 * 2 + c / 2) ^ (g & 2);
          const uint2 v = *reinterpret_cast<const uint2*>(
              st + ((i / 2 * 2 + half) * 8 + g) * 64 + chunk * 16 + c % 2 * 8);
          w[half][0] = v.x, w[half][1] = v.y;
        }
      }
      float p[NT][4] = {};
      const uint4* xg = xs + ((s0 + i) * NT * 2) * 32 + lane;
      uint4 b[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        b[t][0] = xg[t * 64];
        b[t][1] = xg[t * 64 + 32];
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int part = 0; part < C::kParts; ++part) {
          uint32_t a0, a1, a2, a3;
          C::pairs(w[0], s, part, a0, a2);
          C::pairs(w[1], s, part, a1, a3);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4& v = b[t][s / 2];
            mma<AT>(p[t], a0, a1, a2, a3, s % 2 ? v.z : v.x, s % 2 ? v.w : v.y);
          }
        }
      float scale[2], rest[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t v = __shfl_sync(kAll, sb_now[half], (lane & ~3) | i);
        const uint16_t sv = uint16_t(v), bv = uint16_t(v >> 16);
        scale[half] = Act<AT>::to_f32(*reinterpret_cast<const AT*>(&sv));
        rest[half] = fmaf(-C::kUnit, scale[half], Act<AT>::to_f32(*reinterpret_cast<const AT*>(&bv)));
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float2 x =
            *reinterpret_cast<const float2*>(xsum + (s0 + i) * kTokens + 8 * t + 2 * c);
        acc[t][0] = fmaf(scale[0], p[t][0], fmaf(rest[0], x.x, acc[t][0]));
        acc[t][1] = fmaf(scale[0], p[t][1], fmaf(rest[0], x.y, acc[t][1]));
        acc[t][2] = fmaf(scale[1], p[t][2], fmaf(rest[1], x.x, acc[t][2]));
        acc[t][3] = fmaf(scale[1], p[t][3], fmaf(rest[1], x.y, acc[t][3]));
      }
    }
    if (it.stage + 1 < per_item) continue;
    // the item's sums: rows g, g + 8 and tokens 2c, 2c + 1 of each tile from every warp
    float* part = sums + sum_buf * (WK * kTokens * kSumStride);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        part[(wk * kTokens + 8 * t + 2 * c + i % 2) * kSumStride + wn * kRows + 8 * (i / 2) + g] =
            acc[t][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kTokens * kItemRows; i += kThreads) {
      const int tok = i / kItemRows, r = i % kItemRows;
      const int p = pair_of[tile_buf][tok];
      const int64_t row = int64_t(it.block) * kItemRows + r;
      if (p < 0 || row >= a.N) continue;
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < WK; ++k) v += part[(k * kTokens + tok) * kSumStride + r];
      if (a.y_f32)
        static_cast<float*>(a.y)[int64_t(p) * a.N + row] = v;
      else
        static_cast<AT*>(a.y)[int64_t(p) * a.N + row] = Act<AT>::from_f32_rn(v);
    }
    sum_buf ^= 1;  // (a warp that is an item ahead writes the other one)
  }
  copies_wait<0>();
}

size_t shared_bytes(int nt, int wk, int64_t K) {
  const int tokens = 8 * nt;
  return size_t(kWarps) * kRingBytes +
         size_t(2) * wk * tokens * (kRows * (kWarps / wk) + 4) * 4 +
         size_t(K / kGroup) * (tokens * 4 + nt * 1024);
}

constexpr size_t kMostShared = 227 * 1024 - 2560;  // beside first_job and pair_of

template <int BITS, typename AT, int NT, int WK>
qlin_status launch_t(const ExpertArgs& a, unsigned flags, cudaStream_t st) {
  auto kern = stream_kernel<BITS, AT, NT, WK>;
  static std::atomic<unsigned long long> done{0};
  if (!allow_shared(reinterpret_cast<const void*>(kern), int(kMostShared), &done))
    return check_launch("qlin_expert_linear: shared memory");
  const size_t smem = shared_bytes(NT, WK, a.K);
  // tiles of tokens: at most one more than full ones for each expert that has any
  const int64_t used = std::min<int64_t>(a.E, a.n_pairs);
  const int64_t jobs = a.n_pairs / (8 * NT) + used;
  const int64_t rows = kRows * (kWarps / WK);
  const int64_t items = jobs * ((a.N + rows - 1) / rows);
  const int64_t resident = int64_t(sm_count()) * (NT < 4 && smem <= 110 * 1024 ? 2 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(std::min(items, resident)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kern, a);
  return check_launch("qlin_expert_linear");
}

template <int BITS, typename AT, int NT>
qlin_status with_warps(const ExpertArgs& a, unsigned flags, cudaStream_t st) {
  // as many warps to a row as leave each a whole stage
  const int64_t stages = a.K / (kGroup * kGroups);
  if (stages >= 8) return launch_t<BITS, AT, NT, 8>(a, flags, st);
  if (stages >= 4) return launch_t<BITS, AT, NT, 4>(a, flags, st);
  return launch_t<BITS, AT, NT, 2>(a, flags, st);
}

template <int BITS, typename AT>
qlin_status with_tiles(const ExpertArgs& a, int tiles, unsigned flags, cudaStream_t st) {
  if (tiles == 1) return with_warps<BITS, AT, 1>(a, flags, st);
  if (tiles == 2) return with_warps<BITS, AT, 2>(a, flags, st);
  return with_warps<BITS, AT, 4>(a, flags, st);
}

}  // namespace

int expert_stream_tiles(int64_t K, double rows) {
  int tiles = rows <= 2.0 ? 1 : rows <= 8.0 ? 2 : 4;
  while (tiles && shared_bytes(tiles, 8, K) > kMostShared) tiles /= 2;
  return tiles;
}

qlin_status launch_expert_stream(const ExpertArgs& a, int bits, qlin_dtype dtype, int tiles,
                                 unsigned flags, cudaStream_t st) {
  if (dtype == QLIN_F16)
    return bits == 4 ? with_tiles<4, __half>(a, tiles, flags, st)
                     : with_tiles<8, __half>(a, tiles, flags, st);
  return bits == 4 ? with_tiles<4, __nv_bfloat16>(a, tiles, flags, st)
                   : with_tiles<8, __nv_bfloat16>(a, tiles, flags, st);
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
