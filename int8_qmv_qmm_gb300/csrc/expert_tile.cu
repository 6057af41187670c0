// The experts' products where an expert has many rows: tcgen05, as in qmm.cu (128 weight
// rows as the MMA's M, reconstructed into tensor memory as its A operand, a group of 64
// of K to a stage), over the tiles of all experts.
//
// A tile is 128 rows of an expert's weights and up to BN of its tokens.  CTAs, one on an
// SM, walk the list of tiles, a job's (an expert and a stretch of its tokens) row tiles
// one after another, so that those who work on one job share its tokens in L2.
//
// A first kernel copies the tokens' rows in the plan's order to the workspace, so that a
// tile's are neighbours and come as one TMA box a stage; a token's products are written
// to its pair's row.  (Fetching rows from where they are was slower: by TMA gathers of
// four rows, 31 ns each on an SM, 1185 us for 4096 tokens; by cp.async of two or four
// warps 517 and 425; sorted first 304 at the time.)
//
// Both types multiply in f16.  bfloat16 is brought there by powers of two, which the
// outputs are multiplied back by: one for each token (its largest element to 2^14, exact
// down to 2^-28 of it) and one for each weight row, found from its scales and biases, which
// brings the row's largest to 2^14 or more.  Scale and bias are rounded to f16 there, to a
// multiple of 2^-24, and code * scale + bias once more: a weight is off by 2^-11 of it and
// (largest code + 1) * 2^-25 at most, 2^-31 of the row's largest at 8 bits and 2^-35 at 4.
// The first kernel finds the powers.  (Two bfloat16 products for the high and low part of a weight, as
// qmm.cu has them, took 361 us where f16 took 241.)
//
//   warps 0, 2   load the tokens' rows and the packed tiles (TMA, one thread each)
//   warp 1       issues the MMAs, converged, with the operands' descriptors in uniform
//                registers (a loop of one thread alone took 84 cycles an MMA, and set the
//                pace); a tile with fewer tokens than BN multiplies what it has, in steps
//                of 16
//   then         warpgroups that reconstruct stages in turn
//   last         epilogue, two warps for each quarter of the rows: each takes half of the
//                tokens' columns to registers at 16 bits, hands the accumulator back, and
//                stores 16 bytes a lane by way of shared memory while the next tile runs
//                (2 bytes a lane, 64 a warp, took 304 us where this took 271)
//
// 4096 tokens of 8 of 64 experts of 2048 x 2048 at 4 bits (275 GFLOP) take 213 to 221 us by
// machine, 1245 to 1290 TFLOP/s; the same at 8 bits in bfloat16 235.  A stage takes 545 cycles, where the MMAs of a full tile take 538 and the
// reconstructing warps about as long, whatever its columns, of which a fifth is empty;
// 1500 cycles pass between tiles; the copy takes 23 us.  500 tokens of 6
// of 60 experts of 2501 x 1408 at 8 bits (241 MB) take 64 us: a stage of few tokens takes
// the reconstructing warps 410 cycles, where memory would take 180.
//
// Every wait is bounded (about 2 s); one that gives up sets a status bit, and the CTA
// waits for its copies and MMAs in flight, frees its tensor memory and leaves.

#include <algorithm>

#include "expert_plan.cuh"
#include "qmm_core.cuh"

namespace qlin {

__device__ unsigned int g_expert_tile_status = 0;

namespace {

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_expert_tile_status, bit); }

constexpr int kDequantGroups = 2;
constexpr int kDequantWarps = 4 * kDequantGroups;
constexpr int kEpilogueWarps = 8;
constexpr int kFirstDequant = 3;
constexpr int kFirstEpilogue = kFirstDequant + kDequantWarps;
constexpr int kThreads = (kFirstEpilogue + kEpilogueWarps) * 32;
constexpr int kMaxExperts = 512;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxShared = 227 * 1024;
// Tokens whose outputs are turned around in shared memory at a time.
constexpr int kOutTokens = 16;
constexpr int kOutBytes = 2 * 2 * kOutTokens * kBM * 2;  // two for each half

// Three rings with the same index, so that each stage of the way has as many in flight
// as it needs: the tokens' rows and the packed tiles in shared memory, and the A slots in
// tensor memory.  (One ring of five stages for all three held each stage's 36 KB for the
// way of all: 229 us where this takes 213.)
template <int BITS, int BN>
struct Layout {
  static constexpr int kXBytes = BN * kBK * 2;
  static constexpr int kWBytes = Geo<BITS>::kPackedBytes;
  // two accumulators unless they would leave tensor memory too few A slots
  static constexpr int kDBufs = BN >= 256 ? 1 : 2;
  static constexpr int kACol0 = kDBufs * BN;
  static constexpr int kACols = kBK / 2;  // of a slot
  static constexpr int kA = 8;
  static constexpr int kX = BN >= 256 ? 4 : 8;
  static constexpr int kW = 8;
  static constexpr int kRings = kX * kXBytes + kW * kWBytes;
  // barriers and the tensor memory's address, the epilogue's tiles, the plan, the tiles'
  // pairs and factors
  static constexpr int kRestBytes = 512 + kOutBytes + int(sizeof(Jobs<kMaxExperts>)) + 2 * BN * 8;
  static constexpr int kTmemCols = 512;
  static_assert(kACol0 + kA * kACols <= kTmemCols, "");
  // (a barrier of the A ring tells the other two how far the MMAs are; the groups take
  // turns, so that a place of a ring is always the same group's)
  static_assert(kX <= kA && kW % kDequantGroups == 0 && kA % kDequantGroups == 0, "");
  static_assert(1024 + kRings + kRestBytes <= kMaxShared, "");
};

// What the first kernel leaves in the workspace.
struct Sorted {
  uint4* x;           // f16 [n_pairs][K]
  float* token_back;  // [n_pairs] (bfloat16)
  float* row_factor;  // [E][N] (bfloat16)
};
Sorted sorted_in(void* workspace, int64_t n_pairs, int64_t K) {
  uint8_t* p = static_cast<uint8_t*>(workspace);
  Sorted r;
  r.x = reinterpret_cast<uint4*>(p);
  r.token_back = reinterpret_cast<float*>(p + n_pairs * K * 2);
  r.row_factor = r.token_back + n_pairs;
  return r;
}

// True in one lane of a converged warp, which the compiler knows to be one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

constexpr uint64_t kWaitNs = 2000000000ull;

// mbar_wait of a whole warp, converged.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (__all_sync(kAll, ptx::mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(kAll, ptx::mbar_try_wait(bar, parity))) return true;
    if ((i & 63u) == 0 && __any_sync(kAll, ptx::globaltimer_ns() - t0 > limit_ns))
      return false;
  }
}

// Where a CTA is in its list of tiles: a job (an expert and a stretch of its tokens) and
// a block of its weight rows.
struct Tile {
  int job, n_tile, expert;
  int n0, at, count;  // the first weight row, the first token's place in order, tokens
};

// For tests: the producer of packed tiles stops before its stage `stage`, and waits are
// shorter.
struct Stall {
  int stage;
  uint64_t limit_ns;
};

template <int BITS, typename AT, int BN, bool STALL>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                const ExpertArgs a, const Sorted sorted, const Stall stall) {
  const uint64_t limit = STALL ? stall.limit_ns : kWaitNs;
  auto wait = [&](uint32_t bar, uint32_t parity) { return ptx::mbar_wait(bar, parity, limit); };
  auto warp_wait = [&](uint32_t bar, uint32_t parity) { return wait_warp(bar, parity, limit); };
  constexpr bool kHalf = std::is_same<AT, __half>::value;
  using L = Layout<BITS, BN>;
  using G = Geo<BITS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw_base);
  // (what comes from a shuffle the compiler knows to be the same in a warp, and keeps the
  // issuer's loop in uniform registers, as the MMA takes its operands)
  const int warp = __shfl_sync(kAll, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int kb_count = int(a.K) / kBK, N = int(a.N);
  const int n_tiles = (N + kBM - 1) / kBM;

  auto x_addr = [&](int s) { return base + uint32_t(s * L::kXBytes); };
  auto w_addr = [&](int s) { return base + uint32_t(L::kX * L::kXBytes + s * L::kWBytes); };
  const uint32_t bar_base = base + uint32_t(L::kRings);
  auto w_full = [&](int s) { return bar_base + 8u * s; };
  auto w_empty = [&](int s) { return bar_base + 8u * (L::kW + s); };
  // a use's A slot and the tokens' rows are there (one barrier: a wait of the issuer costs
  // what an MMA does)
  auto ready = [&](int s) { return bar_base + 8u * (2 * L::kW + s); };
  // the MMAs of a use have completed: its A slot and its rows are free
  auto done = [&](int s) { return bar_base + 8u * (2 * L::kW + L::kA + s); };
  const uint32_t accf_bar = bar_base + 8u * (2 * L::kW + 2 * L::kA);  // [2]
  const uint32_t acce_bar = accf_bar + 16u;                                    // [2]
  const uint32_t done_bar = acce_bar + 16u;
  static_assert(8 * (2 * L::kW + 2 * L::kA + 5) + 4 <= 508, "barrier block");
  uint8_t* const rest = gbase + L::kRings;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rest + 508);
  uint16_t* turned = reinterpret_cast<uint16_t*>(rest + 512);  // [2][2][kOutTokens][kBM]
  Jobs<kMaxExperts>& plan = *reinterpret_cast<Jobs<kMaxExperts>*>(rest + 512 + kOutBytes);
  const int (&first_job)[kMaxExperts + 1] = plan.first;
  int* pairs = reinterpret_cast<int*>(&plan + 1);             // [2][BN], of the tile's tokens
  float* factors = reinterpret_cast<float*>(pairs + 2 * BN);  // [2][BN] (bfloat16)

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kW; ++s) {
      ptx::mbar_init(w_full(s), 1);
      ptx::mbar_init(w_empty(s), 4);  // the warps of a group
    }
    for (int s = 0; s < L::kA; ++s) {
      ptx::mbar_init(ready(s), 4 + 1);  // the warps of a group and the rows' bytes
      ptx::mbar_init(done(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar + 8u * b, 1);
      ptx::mbar_init(acce_bar + 8u * b, kEpilogueWarps);
    }
    ptx::mbar_init(done_bar, 1);
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tm_x);
    ptx::tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), uint32_t(L::kTmemCols));
    ptx::tmem_relinquish();
  }
  grid_dependency_wait();  // the plan, x and y are the preceding kernels'
  static_assert(kThreads >= kMaxExperts && kThreads / 32 <= 32, "a thread for each expert");
  ptx::tc_fence_before();
  if (fill_jobs(a, BN, plan) && blockIdx.x == 0) report(kStatusPlan);
  ptx::tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(kAll, *tmem_slot, 0);
  // (a kernel that starts from here on finds this one's tensor memory taken already)
  grid_launch_dependents();
  // (from shared memory and without a division: an access to the plan at every tile took
  // each role a thousand cycles)
  const int jobs = __shfl_sync(kAll, first_job[a.E], 0);
  const int step_jobs = int(gridDim.x) / n_tiles, step_tiles = int(gridDim.x) % n_tiles;
  auto fill = [&](Tile& q) {
    while (first_job[q.expert + 1] <= q.job) ++q.expert;
    const int t0 = (q.job - first_job[q.expert]) * BN;
    q.n0 = q.n_tile * kBM;
    q.at = plan.row[q.expert] + t0;
    q.count = min(plan.count[q.expert] - t0, BN);
  };
  auto first_tile = [&] {
    Tile q;
    q.job = int(blockIdx.x) / n_tiles;
    q.n_tile = int(blockIdx.x) - q.job * n_tiles;
    q.expert = 0;
    if (q.job < jobs) fill(q);
    return q;
  };
  auto next_tile = [&](Tile& q) {
    q.job += step_jobs;
    q.n_tile += step_tiles;
    if (q.n_tile >= n_tiles) {
      q.n_tile -= n_tiles;
      ++q.job;
    }
    if (q.job < jobs) fill(q);
  };

  if (warp == 0) {
    // ------------------------------------------------- producer of tokens' rows
    if (lane == 0) {
      int s = 0, u = 0;
      bool ok = true;
      for (Tile q = first_tile(); q.job < jobs && ok; next_tile(q)) {
        // (rows past the tile's tokens are the next expert's, or zeros past the last)
        for (int kb = 0; kb < kb_count; ++kb, ++u) {
          const int before = u - L::kX;  // the use that had the place
          if (before >= 0 &&
              !wait(done(before % L::kA), uint32_t(before / L::kA) & 1u)) {
            report(kStatusWait);
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx(ready(u % L::kA), L::kXBytes);
          ptx::tma_load_2d(x_addr(s), &tm_x, ready(u % L::kA), kb * kBK, q.at);
          if (++s == L::kX) s = 0;
        }
      }
      // (after a wait that gave up: the last loads, one for each place, may be in flight)
      if (!ok)
        for (int v = u > L::kX ? u - L::kX : 0; v < u; ++v)
          if (!wait(ready(v % L::kA), uint32_t(v / L::kA) & 1u)) report(kStatusWait);
    }
  } else if (warp == 2) {
    // ------------------------------------------------- producer of packed tiles
    if (lane == 0) {
      int s = 0, u = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (Tile q = first_tile(); q.job < jobs && ok; next_tile(q)) {
        const int row = q.expert * N + q.n0;
        for (int kb = 0; kb < kb_count; ++kb, ++u) {
          if (STALL && u == stall.stage) {
            ok = false;
            break;
          }
          if (u >= L::kW && !wait(w_empty(s), phase ^ 1u)) {
            report(kStatusWait);
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx(w_full(s), L::kWBytes);
          ptx::tma_load_2d(w_addr(s), &tm_w, w_full(s), kb * G::kWordsPerGroup, row);
          if (++s == L::kW) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok)
        for (int v = 0; v < L::kW && v < u; ++v) {
          if (--s < 0) {
            s = L::kW - 1;
            phase ^= 1u;
          }
          if (!wait(w_full(s), phase)) report(kStatusWait);
        }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    const bool leads = elect_one();
    const uint64_t b_desc0 = ptx::sw128_kmajor_desc(base);
    int s = 0, xs = 0, i = 0;
    uint32_t phase = 0;
    bool ok = true, any = false;
    for (Tile q = first_tile(); q.job < jobs && ok; next_tile(q), ++i) {
      const uint32_t columns = uint32_t(__shfl_sync(kAll, (q.count + 15) & ~15, 0));
      const uint32_t idesc = ptx::idesc_f16(0u, kBM, columns);
      const int buf = i % L::kDBufs;
      if (i >= L::kDBufs &&
          !warp_wait(acce_bar + 8u * buf, uint32_t(i / L::kDBufs - 1) & 1u)) {
        report(kStatusWait);
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t d_tmem = tmem_base + uint32_t(buf * BN);
      uint32_t more = 0;
      for (int kb = 0; kb < kb_count; ++kb) {
        if (!warp_wait(ready(s), phase)) {
          report(kStatusWait);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t a_tmem = tmem_base + uint32_t(L::kACol0 + s * L::kACols);
        const uint64_t bd = b_desc0 + uint64_t(uint32_t(xs * L::kXBytes) >> 4);
        if (leads) {
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            mma_f16_ts(d_tmem, a_tmem + uint32_t(8 * kk), bd + uint64_t(2 * kk), idesc,
                       kk > 0 ? 1u : more);
          }
          ptx::mma_commit(done(s));
        }
        __syncwarp();
        more = 1;
        any = true;
        if (++s == L::kA) {
          s = 0;
          phase ^= 1u;
        }
        if (++xs == L::kX) xs = 0;
      }
      if (ok && leads) ptx::mma_commit(accf_bar + 8u * buf);
      __syncwarp();
    }
    // before tensor memory is freed every MMA issued here must have completed (a CTA that
    // issued none commits nothing: nobody would wait for that arrival, and it could come
    // after the CTA has left, in the barriers of the next one)
    if (any && leads) ptx::mma_commit(done_bar);
    __syncwarp();
    if (any && !wait(done_bar, 0)) report(kStatusWait);
    __syncwarp();
  } else if (warp < kFirstEpilogue) {
    // -------------------------------- reconstruct (the warpgroups in turn)
    const int grp = (warp - kFirstDequant) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // weight row within the tile
    const uint32_t a_lane = tmem_base + (uint32_t(quarter * 32) << 16) + uint32_t(L::kACol0);
    int u = grp;  // the group's next use
    int ws = grp, as = grp;
    uint32_t w_phase = 0, a_phase = 0;
    int kb0 = grp;  // its first stage of the tile
    bool ok = true;
    for (Tile q = first_tile(); q.job < jobs && ok; next_tile(q)) {
      const int n = q.n0 + r;
      const bool row_ok = n < N;
      const int64_t at = (int64_t(q.expert) * N + min(n, N - 1)) * kb_count;
      const AT* srow = static_cast<const AT*>(a.scales) + at;
      const AT* brow = static_cast<const AT*>(a.biases) + at;
      float factor = 1.f;
      if constexpr (!kHalf) factor = sorted.row_factor[int64_t(q.expert) * N + min(n, N - 1)];
      int kb = kb0;
      AT next_sc, next_bc;  // (a stage ahead: their way is longer than a stage)
      if (kb < kb_count) {
        next_sc = srow[kb];
        next_bc = brow[kb];
      }
      for (; kb < kb_count; kb += kDequantGroups, u += kDequantGroups) {
        const AT sc = next_sc, bc = next_bc;
        if (kb + kDequantGroups < kb_count) {
          next_sc = srow[kb + kDequantGroups];
          next_bc = brow[kb + kDequantGroups];
        }
        if (!warp_wait(w_full(ws), w_phase)) {
          report(kStatusWait);
          ok = false;
          break;
        }
        const uint8_t* wrow = gbase + (w_addr(ws) - base) + r * G::kPackedRowBytes;
        __half scale, bias;
        if constexpr (kHalf) {
          scale = sc;
          bias = bc;
        } else {
          scale = __float2half_rn(Act<AT>::to_f32(sc) * factor);
          bias = __float2half_rn(Act<AT>::to_f32(bc) * factor);
        }
        uint32_t w[32], none[1];
        dequant_row<BITS, __half, 1>(wrow, r, scale, bias, row_ok, w, none);
        // the A slot's last products
        if (u >= L::kA && !warp_wait(done(as), a_phase ^ 1u)) {
          report(kStatusWait);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        tmem_st_32x32b_x32(a_lane + uint32_t(as * L::kACols), w);
        tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        // (the packed tile's place is free only here, where what was read from it has been
        // stored: an arrival straight after the loads can come before they are done, while
        // scattered loads of scales hold them up, and the next tile be read in their place)
        if (lane == 0) {
          ptx::mbar_arrive(w_empty(ws));
          ptx::mbar_arrive(ready(as));
        }
        if ((ws += kDequantGroups) >= L::kW) {
          ws = grp;
          w_phase ^= 1u;
        }
        if ((as += kDequantGroups) >= L::kA) {
          as = grp;
          a_phase ^= 1u;
        }
      }
      kb0 = kb - kb_count;  // (the turns go on from tile to tile)
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - kFirstEpilogue) >> 2;
    const int et = (threadIdx.x - kFirstEpilogue * 32) & 127;  // within the half
    constexpr int kCols = BN / 2;                              // of a half
    static_assert(kCols % (2 * kOutTokens) == 0, "the tiles take turns");
    const bool wide = N % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
    auto half_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); };
    bool live = true;
    int i = 0;
    for (Tile q = first_tile(); q.job < jobs; next_tile(q), ++i) {
      int* mine = pairs + (i & 1) * BN + half * kCols;
      float* back = factors + (i & 1) * BN + half * kCols;
      const int count = min(q.count - half * kCols, kCols);  // tokens of the half
      for (int j = et; j < kCols; j += 128) {
        int p = -1;
        if (j < count) {
          const int at = q.at + half * kCols + j;
          p = a.order[at];
          if (p < 0 || p >= a.n_pairs) {
            report(kStatusPlan);
            p = -1;
          }
          if constexpr (!kHalf) back[j] = sorted.token_back[at];
        }
        mine[j] = p;
      }
      const int n = q.n0 + quarter * 32 + lane;
      float row_back = 1.f;
      if constexpr (!kHalf)
        row_back = 1.f / sorted.row_factor[int64_t(q.expert) * N + min(n, N - 1)];
      // (two lists: nobody is still at the one before the last)
      half_sync();
      const int buf = i % L::kDBufs;
      // (a warp whose wait gave up stores nothing from there on, but comes to every barrier:
      // the other warps of its half wait there without a limit)
      if (live && !warp_wait(accf_bar + 8u * buf, uint32_t(i / L::kDBufs) & 1u)) {
        report(kStatusWait);
        live = false;
      }
      ptx::tc_fence_after();
      const uint32_t t_lane = tmem_base + (uint32_t(quarter * 32) << 16) +
                              uint32_t(buf * BN + half * kCols);
      auto hand_back = [&] {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(acce_bar + 8u * buf);
      };
      // sixteen tokens' sums, as they are or (bfloat16) multiplied back
      auto load = [&](int c, float (&f)[16]) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(t_lane + uint32_t(c), v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          f[j] = __uint_as_float(v[j]);
          if constexpr (!kHalf) f[j] = f[j] * row_back * back[c + j];
        }
      };
      if (a.y_f32) {
#pragma unroll 1
        for (int c = 0; c < count; c += 16) {
          float f[16];
          load(c, f);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int p = mine[c + j];  // (-1 past the last token)
            if (live && n < N && p >= 0) static_cast<float*>(a.y)[int64_t(p) * N + n] = f[j];
          }
        }
        hand_back();
        continue;
      }
      uint32_t out[kCols / 2];  // two tokens each
#pragma unroll
      for (int c = 0; c < kCols; c += 32) {
        if (c < count) {
          uint32_t v[32];  // (two loads, one wait)
          ptx::tmem_ld_32x32b_x16(t_lane + uint32_t(c), *reinterpret_cast<uint32_t(*)[16]>(v));
          ptx::tmem_ld_32x32b_x16(t_lane + uint32_t(c + 16), *reinterpret_cast<uint32_t(*)[16]>(v + 16));
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float x = __uint_as_float(v[2 * j]), y = __uint_as_float(v[2 * j + 1]);
            if constexpr (!kHalf) {
              x = x * row_back * back[c + 2 * j];
              y = y * row_back * back[c + 2 * j + 1];
            }
            typename Act<AT>::T2 h;
            h.x = Act<AT>::from_f32_rn(x);
            h.y = Act<AT>::from_f32_rn(y);
            out[c / 2 + j] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
      }
      hand_back();
      if (wide) {
        // by way of shared memory, so that 16 lanes store a token's 128 outputs
#pragma unroll
        for (int c = 0; c < kCols; c += kOutTokens) {
          if (c < count) {
            uint16_t* tile = turned + (half * 2 + (c / kOutTokens & 1)) * (kOutTokens * kBM);
#pragma unroll
            for (int j = 0; j < kOutTokens; j += 2) {
              const uint32_t v = out[(c + j) / 2];
              tile[j * kBM + quarter * 32 + lane] = uint16_t(v);
              tile[(j + 1) * kBM + quarter * 32 + lane] = uint16_t(v >> 16);
            }
            // (who fills a tile again has passed the other's barrier since)
            half_sync();
            const int n8 = et % 16 * 8;
#pragma unroll
            for (int j = 0; j < kOutTokens; j += 8) {
              const int p = mine[c + j + et / 16];
              if (live && p >= 0 && q.n0 + n8 < N)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + int64_t(p) * N + q.n0 +
                                          n8) =
                    *reinterpret_cast<const uint4*>(tile + (j + et / 16) * kBM + n8);
            }
          }
        }
      } else if (live && n < N) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + n;
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          if (c < count) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int p = mine[c + j];
              const uint32_t v = out[(c + j) / 2];
              if (p >= 0) y[int64_t(p) * N] = uint16_t(j % 2 ? v >> 16 : v);
            }
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, uint32_t(L::kTmemCols));
  }
}

// ------------------------------------------------------------------- rows in order
constexpr int kSortWarps = 8;
constexpr int kRowsAWarp = 8;  // weight rows whose factor a warp finds at a time

// The power of two that brings a magnitude of these float bits to 2^14 .. 2^15; for none
// (0, or not finite) 1.  Below 2^-100 it stays at 2^114.
__device__ __forceinline__ float factor_for(uint32_t bits) {
  const int e = int(bits >> 23);
  const int up = e == 255 || bits == 0u ? 127 : e < 27 ? 127 + 114 : 127 + 14 + 127 - e;
  return __uint_as_float(uint32_t(up) << 23);
}

// The rows of x in the plan's order, a warp a row (pairs that are none left out), and for
// bfloat16, in f16 by their factors, whose inverses go to token_back; further CTAs find
// the factors of the weight rows.
template <typename AT>
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_rows_kernel(const ExpertArgs a, const Sorted out, int64_t row_ctas, int qmax) {
  constexpr bool kHalf = std::is_same<AT, __half>::value;
  const int lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  if (!kHalf && blockIdx.x >= row_ctas) {
    // a weight is between its group's bias and bias + qmax * scale
    const int64_t row = ((int64_t(blockIdx.x) - row_ctas) * kSortWarps + (threadIdx.x >> 5)) *
                            kRowsAWarp + lane / 4;
    if (row >= int64_t(a.E) * a.N) return;
    const int groups = int(a.K) / kGroup;
    const AT* s = static_cast<const AT*>(a.scales) + row * groups;
    const AT* b = static_cast<const AT*>(a.biases) + row * groups;
    uint32_t most = 0u;
#pragma unroll 4
    for (int g = lane % 4; g < groups; g += 4) {
      const float low = Act<AT>::to_f32(b[g]);
      const float high = fmaf(float(qmax), Act<AT>::to_f32(s[g]), low);
      most = max(most, max(__float_as_uint(fabsf(low)), __float_as_uint(fabsf(high))));
    }
    // (the four lanes of a row leave together)
    const unsigned mask = 15u << (lane & ~3);
    for (int d = 1; d < 4; d <<= 1) most = max(most, __shfl_xor_sync(mask, most, d));
    if (lane % 4 == 0) out.row_factor[row] = factor_for(most);
    return;
  }
  const int64_t i = int64_t(blockIdx.x) * kSortWarps + (threadIdx.x >> 5);
  if (i >= a.n_pairs) return;
  const int p = a.order[i];
  if (p < 0 || p >= a.n_pairs) return;
  const int packs = int(a.K) / 8;
  const uint4* from =
      reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) +
                                     int64_t(p / a.pairs_per_row) * a.x_stride);
  uint4* to = out.x + i * packs;
  float factor = 1.f;
  if constexpr (!kHalf) {
    uint32_t most = 0u;  // magnitudes' bits, two at a time
#pragma unroll 4
    for (int k = lane; k < packs; k += 32) {
      const uint4 v = from[k];
      most = __vmaxu2(most, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    most = max(most & 0xffffu, most >> 16) << 16;
    most = __reduce_max_sync(kAll, most);
    factor = factor_for(most);
    if (lane == 0) out.token_back[i] = 1.f / factor;
  }
  // four loads before the first store
  for (int k0 = lane; k0 < packs; k0 += 128) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k0 + 32 * j < packs) v[j] = from[k0 + 32 * j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!kHalf) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 h = __floats2half2_rn(__uint_as_float(w[e] << 16) * factor,
                                              __uint_as_float(w[e] & 0xffff0000u) * factor);
          w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      if (k0 + 32 * j < packs) to[k0 + 32 * j] = v[j];
    }
  }
}

template <int BITS, typename AT, int BN, bool STALL = false>
qlin_status launch_t(const ExpertArgs& a, unsigned flags, cudaStream_t st, Stall stall = {}) {
  using L = Layout<BITS, BN>;
  constexpr int kBytes = 1024 + L::kRings + L::kRestBytes;
  auto kern = tile_kernel<BITS, AT, BN, STALL>;
  static std::atomic<unsigned long long> done{0};
  if (!allow_shared(reinterpret_cast<const void*>(kern), kBytes, &done))
    return check_launch("qlin_expert_linear: shared memory");
  const int64_t words = a.K * BITS / 32;
  CUtensorMap tm_x, tm_w;
  const Sorted sorted = sorted_in(a.workspace, a.n_pairs, a.K);
  qlin_status s = make_map(&tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, sorted.x, uint64_t(a.K), uint64_t(a.n_pairs),
                           uint64_t(a.K) * 2, kBK, BN, CU_TENSOR_MAP_SWIZZLE_128B);
  if (s != QLIN_OK) return s;
  s = make_map(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.wq, uint64_t(words),
               uint64_t(a.E) * uint64_t(a.N), uint64_t(words) * 4, Geo<BITS>::kWordsPerGroup, kBM,
               BITS == 4 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B);
  if (s != QLIN_OK) return s;
  const int64_t jobs = a.n_pairs / BN + std::min<int64_t>(a.E, a.n_pairs);
  const int64_t tiles = jobs * ((a.N + kBM - 1) / kBM);
  if (tiles > (int64_t(1) << 30))
    return fail(QLIN_ERR_UNSUPPORTED, "qlin_expert_linear: too many tiles");
  cudaLaunchConfig_t cfg = {};
  const int64_t row_ctas = (a.n_pairs + kSortWarps - 1) / kSortWarps;
  const int64_t at_once = kSortWarps * kRowsAWarp;
  const int64_t factor_ctas =
      std::is_same<AT, __half>::value ? 0 : (int64_t(a.E) * a.N + at_once - 1) / at_once;
  cfg.gridDim = dim3(unsigned(row_ctas + factor_ctas));
  cfg.blockDim = dim3(kSortWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, sort_rows_kernel<AT>, a, sorted, row_ctas, (1 << BITS) - 1) !=
      cudaSuccess)
    return check_launch("qlin_expert_linear");
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(tiles, sm_count())));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kern, tm_x, tm_w, a, sorted, stall);
  return check_launch("qlin_expert_linear");
}

template <int BITS, typename AT>
qlin_status dispatch(const ExpertArgs& a, double rows, unsigned flags, cudaStream_t st) {
  if (rows <= 64.0) return launch_t<BITS, AT, 64>(a, flags, st);
  if (rows <= 128.0) return launch_t<BITS, AT, 128>(a, flags, st);
  return launch_t<BITS, AT, 256>(a, flags, st);
}

}  // namespace

qlin_status launch_expert_tile(const ExpertArgs& a, int bits, qlin_dtype dtype, double rows,
                               unsigned flags, cudaStream_t st) {
  if (dtype == QLIN_F16)
    return bits == 4 ? dispatch<4, __half>(a, rows, flags, st)
                     : dispatch<8, __half>(a, rows, flags, st);
  return bits == 4 ? dispatch<4, __nv_bfloat16>(a, rows, flags, st)
                   : dispatch<8, __nv_bfloat16>(a, rows, flags, st);
}

qlin_status launch_expert_stalled(const ExpertArgs& a, int stage, unsigned wait_limit_us,
                                  cudaStream_t st) {
  return launch_t<4, __half, 64, true>(a, 0, st, Stall{stage, uint64_t(wait_limit_us) * 1000});
}

size_t expert_tile_workspace_size(int64_t n_pairs, int E, int64_t N, int64_t K) {
  return size_t(n_pairs) * K * 2 + size_t(n_pairs + int64_t(E) * N) * 4;
}

cudaError_t expert_tile_take_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_expert_tile_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_expert_tile_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace qlin
