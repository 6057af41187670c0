// Attention of slots with few new rows: single tokens, drafts, short chunks.
//
// What bounds it is reading the cache once, so the blocks of all slots, heads
// and row tiles are put in one list and every team of warps takes an equal,
// consecutive share of it, however long or short the slots are.  Inside its
// share a team's warps take the blocks in turn.  Each warp streams its blocks
// through a ring of its own in shared memory (bulk copies, one for the keys and
// one for the values of a block), so no barrier stands in its loop; the page
// numbers and scales of its next 32 blocks are fetched at once, a lane each.
//
// A piece is what a team has of one tile (slot, key/value head, 16 rows).  At
// its end the warps' sums are joined through shared memory.  A tile that lies
// in one team's share is written out; else the team leaves its part in the
// workspace, and the team that finds itself last joins the parts, always in the
// list's order: the result does not depend on which came last.

#include "attention_core.cuh"
#include "sm100_ptx.cuh"

namespace qlin {
namespace attention {

__device__ unsigned int g_split_status = 0;

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRingBytes = 16384;  // of a warp
constexpr int kMaxSlots = 2048;
constexpr int kInfo = 8;           // blocks that the copies may run ahead

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_split_status, bit); }

// Copies `bytes` from global memory to dst, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  ptx::mbar_arrive_expect_tx(bar, bytes);
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

struct Info {  // of a block that is being copied
  float k_scale, v_scale;
  int kind;
};
enum { kCodes = 0, kTail = 1, kNone = 2 };

// NT: tiles of 8 rows that a warp takes at once.
template <int D, int NT>
struct Layout {
  static constexpr int kRows = 8 * NT;
  static constexpr int kChunk = kBlock * D;             // bytes of a block's keys or values
  static constexpr int kRing = kRingBytes / kChunk;     // chunks in a warp's ring
  static constexpr int kOut = D + 4;                    // floats of a joined row
  static constexpr int kRingAt = 0;
  static constexpr int kOutAt = kWarps * kRingBytes;
  static constexpr int kStatAt = kOutAt + kWarps * kRows * kOut * 4;  // m and l
  static constexpr int kInfoAt = kStatAt + 2 * kWarps * kRows * 4;
  static constexpr int kBarAt = kInfoAt + kWarps * kInfo * int(sizeof(Info));
  static constexpr int kScanAt = (kBarAt + kWarps * kRing * 8 + 15) / 16 * 16;
  static constexpr int kListAt = kScanAt + 2 * kWarps * 8 + 16;
  static int bytes(int slots) { return kListAt + (slots + 1) * 8 + slots * 4; }
  // the workspace: a part is kRows rows of D sums, then their m and l
  static constexpr int kPart = kRows * (D + 2);  // floats
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) split_kernel(const Args a, float* parts,
                                                            unsigned* counters) {
  using L = Layout<D, NT>;
  constexpr int kRows = L::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_out = reinterpret_cast<float*>(smem + L::kOutAt);
  float* s_m = reinterpret_cast<float*>(smem + L::kStatAt);
  float* s_l = s_m + kWarps * kRows;
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + L::kScanAt);
  int* s_last = reinterpret_cast<int*>(smem + L::kScanAt + 2 * kWarps * 8);  // of a team: 4
  int64_t* s_list = reinterpret_cast<int64_t*>(smem + L::kListAt);  // blocks before each slot
  int32_t* s_total = reinterpret_cast<int32_t*>(s_list + a.c.slots + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + L::kRingAt + warp * kRingBytes;
  Info* info = reinterpret_cast<Info*>(smem + L::kInfoAt) + warp * kInfo;
  const uint32_t bar = ptx::smem_u32(smem + L::kBarAt) + warp * L::kRing * 8;
  if (lane == 0)
    for (int i = 0; i < L::kRing; ++i) ptx::mbar_init(bar + 8 * i, 1);
  ptx::fence_mbar_init();
  grid_launch_dependents();
  grid_dependency_wait();

  // the list: blocks before each slot, and how many tiles there are in all
  int64_t blocks = 0, tiles = 0;
  for (int b0 = 0; b0 < a.c.slots; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int64_t mine = 0, pieces = 0;
    if (b < a.c.slots) {
      const SlotRows r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
      const int64_t rows = int64_t(r.n) * a.group;
      if (blockIdx.x == 0) {
        if (r.bad) report(kStatusRows);
        if (r.n > a.max_new) report(kStatusMaxNew);
      }
      s_total[b] = r.held + r.n;
      if (rows <= kSplitRows) pieces = (rows + kRows - 1) / kRows * a.c.kv_heads;
      mine = pieces * ((r.held + r.n + kBlock - 1) / kBlock);
    }
    int64_t upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    for (int d = 16; d; d >>= 1) pieces += __shfl_xor_sync(0xffffffffu, pieces, d);
    __syncthreads();
    if (lane == 31) {
      s_scan[warp] = upto;
      s_scan[kWarps + warp] = pieces;
    }
    __syncthreads();
    int64_t before = blocks;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += s_scan[i];
      blocks += s_scan[i];
      tiles += s_scan[kWarps + i];
    }
    if (b < a.c.slots) s_list[b] = before + upto - mine;
  }
  if (threadIdx.x == 0) s_list[a.c.slots] = blocks;
  __syncthreads();
  if (blocks == 0) return;

  // Teams: as many warps to a tile as there are warps for it, so that tiles are
  // cut only where they have to be; and no team without a block for each warp,
  // unless that left tiles without a team.
  const int64_t all_warps = int64_t(gridDim.x) * kWarps;
  int64_t each = all_warps / tiles;
  each = each < blocks / tiles ? each : blocks / tiles;
  const int team_warps = each >= 8 ? 8 : each >= 4 ? 4 : each >= 2 ? 2 : 1;
  int64_t teams = all_warps / team_warps, useful = blocks / team_warps;
  useful = useful > tiles ? useful : tiles;
  teams = teams < useful ? teams : useful;
  teams = teams < blocks ? teams : blocks;
  // team i of a CTA: spread over the CTAs first
  const int in_cta = warp / team_warps, member = warp % team_warps;
  const int64_t team = int64_t(in_cta) * gridDim.x + blockIdx.x;
  if (team >= teams) return;  // (a team's warps leave together; barriers are the teams')
  const int team_threads = team_warps * 32;
  auto team_barrier = [&] {
    if (team_warps == 1)
      __syncwarp();
    else
      named_barrier(1 + in_cta, team_threads);
  };
  auto start_of = [&](int64_t i) { return i * blocks / teams; };
  auto team_of = [&](int64_t x) { return ((x + 1) * teams - 1) / blocks; };
  const int64_t x0 = start_of(team), x1 = start_of(team + 1);
  const int64_t count = x1 - x0 > member ? (x1 - x0 - member + team_warps - 1) / team_warps : 0;

  // where block x of the list lies
  auto slot_at = [&](int64_t x) {
    int lo = 0, hi = a.c.slots;  // s_list[lo] <= x < s_list[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_list[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };

  // ---- the copies of this warp's blocks x0 + member, + team_warps, ...
  int64_t next = 0;      // the next block to copy
  bool keys_sent = false;
  unsigned sent = 0, used = 0;  // chunks
  int64_t done = 0;      // blocks that are through
  const uint8_t* my_src = nullptr;  // of lane l: block (next / 32 * 32 + l)
  float2 my_scales = make_float2(0.f, 0.f);
  int my_kind = kNone;
  auto pump = [&] {
    while (next < count && sent - used < unsigned(L::kRing) && next - done < kInfo) {
      if (!keys_sent && (next & 31) == 0) {
        const int64_t i = next + lane;
        my_kind = kNone;
        if (i < count) {
          const int64_t x = x0 + member + i * team_warps;
          const int b = slot_at(x);
          const int total = s_total[b], n = (total + kBlock - 1) / kBlock;
          const int64_t in_slot = x - s_list[b];
          const int j = int(in_slot % n);
          const int64_t rows = int64_t(a.starts[b + 1] - a.starts[b]) * a.group;
          const int kvh = int(in_slot / n / ((rows + kRows - 1) / kRows));
          if (j >= total / kBlock) {
            my_kind = kTail;
          } else {
            const int64_t page = page_of(a.c, b, j);
            if (page < 0) {
              report(kStatusPage);
            } else {
              const int64_t at = page * a.c.kv_heads + kvh;
              my_kind = kCodes;
              my_src = static_cast<const uint8_t*>(a.c.pages) + at * 2 * L::kChunk;
              my_scales = reinterpret_cast<const float2*>(a.c.scales)[at];
            }
          }
        }
      }
      const int from = int(next & 31);
      const int kind = __shfl_sync(0xffffffffu, my_kind, from);
      const float ks = __shfl_sync(0xffffffffu, my_scales.x, from);
      const float vs = __shfl_sync(0xffffffffu, my_scales.y, from);
      const uint8_t* src = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(my_src), from));
      if (!keys_sent && lane == 0) info[next % kInfo] = Info{ks, vs, kind};
      if (kind != kCodes) {
        ++next;
        continue;
      }
      const unsigned slot = sent % L::kRing;
      if (lane == 0)
        bulk_load(ptx::smem_u32(ring + slot * L::kChunk), src + (keys_sent ? L::kChunk : 0),
                  L::kChunk, bar + 8 * slot);
      ++sent;
      next += keys_sent;
      keys_sent = !keys_sent;
    }
    __syncwarp();
  };
  // the next chunk, when it has landed
  auto chunk = [&]() -> const uint8_t* {
    const unsigned slot = used % L::kRing;
    if (!ptx::mbar_wait(bar + 8 * slot, (used / L::kRing) & 1) && lane == 0) report(kStatusWait);
    return ring + slot * L::kChunk;
  };
  auto release = [&] {
    __syncwarp();  // every lane has read it
    ++used;
    pump();
  };
  pump();

  Warp<T, D, NT> w;
  for (int64_t x = x0; x < x1;) {
    // ---- a piece: blocks x .. end of the tile that x is in
    const int b = slot_at(x);
    const SlotRows r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
    const int rows = r.n * a.group, n = (r.held + r.n + kBlock - 1) / kBlock;
    const int64_t in_slot = x - s_list[b], tile = in_slot / n;
    const int row_tiles = (rows + kRows - 1) / kRows;
    const int kvh = int(tile / row_tiles), row0 = int(tile % row_tiles) * kRows;
    const int64_t first = x - in_slot % n, last = first + n;  // the tile's blocks in the list
    const int64_t end = last < x1 ? last : x1;
    const bool over = r.n > a.max_new;
    const int here = min(kRows, rows - row0);
    const T* qp[NT];
    int pos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + 8 * n + g;
      qp[n] = row < rows ? static_cast<const T*>(a.q) + (r.row0 + row / a.group) * a.q_stride +
                               (kvh * a.group + row % a.group) * D
                         : nullptr;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int mine = row0 + 8 * n + 2 * t + i;
        pos[n][i] = mine < rows ? r.held + mine / a.group : -1;
      }
    }
    w.init();
    w.load_q(qp, a.scale_log2, lane);
    const int first_pos = r.held + row0 / a.group;
    for (; done < count; ++done) {
      const int64_t at = x0 + member + done * team_warps;
      if (at >= end) break;
      const int j = int(at - first);
      const Info f = info[done % kInfo];
      int seen[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        seen[n][0] = pos[n][0] - j * kBlock + 1, seen[n][1] = pos[n][1] - j * kBlock + 1;
      if (f.kind == kCodes) {
        const bool mask = first_pos < j * kBlock + kBlock - 1;
        float s[4][NT][4];
        uint32_t p[4][NT][2];
        w.scores(chunk(), s, lane);
        release();
        w.probabilities(s, p, f.k_scale, f.v_scale, seen, mask, lane);
        w.values(chunk(), p, lane);
        release();
      } else if (f.kind == kTail) {
        w.tail(static_cast<const T*>(a.c.tail) +
                   (int64_t(b) * a.c.kv_heads + kvh) * 2 * kBlock * D,
               r.held + r.n - j * kBlock, qp, a.scale_log2, seen, lane);
      }
    }
    pump();  // (blocks without copies at the piece's end)

    // ---- join the team's warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * n + 2 * t + i;
        float l = w.l[n][i];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) {
          s_m[warp * kRows + row] = w.m[n][i];
          s_l[warp * kRows + row] = l;
        }
        if (row < here) {
          float* dst = s_out + (warp * kRows + row) * L::kOut + g;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            dst[16 * c] = w.o[c][n][i] * w.unit;
            dst[16 * c + 8] = w.o[c][n][2 + i] * w.unit;
          }
        }
      }
    team_barrier();
    const bool whole = x == first && end == last;
    const int w0 = warp - member, mine = member * 32 + lane;
    float* part = parts + (2 * team + (x == first ? 1 : 0)) * L::kPart;
    T* out = static_cast<T*>(a.out);
    auto store = [&](int row, int d, float4 o, float sum) {
      const float inv = sum > 0.f && !over ? 1.f / sum : 0.f;
      const int rr = row0 + row;
      T* dst = out + ((r.row0 + rr / a.group) * a.q_heads + kvh * a.group + rr % a.group) * D + d;
      union {
        T v[4];
        uint2 bits;
      } u;
      u.v[0] = Act<T>::from_f32_rn(over ? 0.f : o.x * inv);
      u.v[1] = Act<T>::from_f32_rn(over ? 0.f : o.y * inv);
      u.v[2] = Act<T>::from_f32_rn(over ? 0.f : o.z * inv);
      u.v[3] = Act<T>::from_f32_rn(over ? 0.f : o.w * inv);
      *reinterpret_cast<uint2*>(dst) = u.bits;
    };
    for (int i = mine; i < here * (D / 4); i += team_threads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float top = -INFINITY;
      for (int k = w0; k < w0 + team_warps; ++k) top = fmaxf(top, s_m[k * kRows + row]);
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = w0; k < w0 + team_warps; ++k) {
        const float m = s_m[k * kRows + row];
        const float f = m == -INFINITY ? 0.f : exp2_fast(m - top);
        const float4 v = *reinterpret_cast<const float4*>(s_out + (k * kRows + row) * L::kOut + d);
        sum += s_l[k * kRows + row] * f;
        o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
      }
      if (whole) {
        store(row, d, o, sum);
      } else {
        __stcg(reinterpret_cast<float4*>(part + row * D + d), o);
        if (d == 0) {
          __stcg(part + kRows * D + row, top);
          __stcg(part + kRows * D + kRows + row, sum);
        }
      }
    }
    if (!whole) {
      const int64_t t0 = team_of(first), t1 = team_of(last - 1);
      __threadfence();
      team_barrier();
      if (mine == 0) {
        const unsigned before = atomicAdd(counters + t0, 1u);
        const bool is_last = before == unsigned(t1 - t0);
        if (is_last) atomicExch(counters + t0, 0u);  // as it was, for the next call
        s_last[in_cta] = is_last;
      }
      team_barrier();
      if (s_last[in_cta]) {
        __threadfence();
        for (int i = mine; i < here * (D / 4); i += team_threads) {
          const int row = i / (D / 4), d = i % (D / 4) * 4;
          // a running join: parts come in the list's order
          float top = -INFINITY, sum = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int64_t k = t0; k <= t1; ++k) {
            const float* from = parts + (2 * k + (k == t0 ? 1 : 0)) * L::kPart;
            const float m = __ldcg(from + kRows * D + row);
            const float l = __ldcg(from + kRows * D + kRows + row);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(from + row * D + d));
            const float next_top = fmaxf(top, m);
            const float base = next_top == -INFINITY ? 0.f : next_top;
            const float f0 = exp2_fast(top - base), f1 = exp2_fast(m - base);
            sum = sum * f0 + l * f1;
            o.x = o.x * f0 + v.x * f1, o.y = o.y * f0 + v.y * f1;
            o.z = o.z * f0 + v.z * f1, o.w = o.w * f0 + v.w * f1;
            top = next_top;
          }
          store(row, d, o, sum);
        }
      }
    }
    team_barrier();  // the joined rows are read before the next piece writes its own
    x = end;
  }
}

template <typename T, int D, int NT>
void launch_t(const Args& a, void* workspace, unsigned flags, cudaStream_t st) {
  using L = Layout<D, NT>;
  static_assert(L::kListAt + (kMaxSlots + 1) * 8 + kMaxSlots * 4 <= 227 * 1024, "it fits");
  if (cudaFuncSetAttribute(split_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           L::bytes(kMaxSlots)) != cudaSuccess)
    return;  // (the caller's check of the launch reports it)
  const int sms = sm_count();
  unsigned* counters = static_cast<unsigned*>(workspace);
  float* parts = reinterpret_cast<float*>(counters + (sms * kWarps + 63) / 64 * 64);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(L::bytes(a.c.slots));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, split_kernel<T, D, NT>, a, parts, counters);
}

template <typename T, int D>
void launch_rows(const Args& a, void* workspace, unsigned flags, cudaStream_t st) {
  if (int64_t(a.max_new) * a.group <= 8)
    launch_t<T, D, 1>(a, workspace, flags, st);
  else
    launch_t<T, D, 2>(a, workspace, flags, st);
}

}  // namespace

size_t split_workspace_size(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  const size_t teams = size_t(sm_count()) * kWarps;
  return (teams + 63) / 64 * 64 * 4 + teams * 2 * 16 * (head_dim + 2) * 4;
}

void launch_split(const Args& a, void* workspace, unsigned flags, cudaStream_t st) {
  if (a.c.dtype == QLIN_F16)
    a.c.head_dim == 64 ? launch_rows<__half, 64>(a, workspace, flags, st)
                       : launch_rows<__half, 128>(a, workspace, flags, st);
  else
    a.c.head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(a, workspace, flags, st)
                       : launch_rows<__nv_bfloat16, 128>(a, workspace, flags, st);
}

cudaError_t split_take_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_split_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_split_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace attention
}  // namespace qlin
