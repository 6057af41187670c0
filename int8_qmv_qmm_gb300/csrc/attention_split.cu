// Attention of slots with few new rows: single tokens, drafts, short chunks.
//
// What bounds it is reading the cache once, so the blocks of all slots, heads
// and row tiles are put in one list and every warp takes an equal, consecutive
// share of it, however long or short the slots are.  One sequence of 131071
// tokens, 8 heads of 128 (269 MB): 50 us, 5.4 TB/s, and 60 with the join; 32 of up
// to 8192, 8 heads of 64 (185 MB): 42 us, 4.4 TB/s, and 49.  There a block's
// instructions (the widening of its codes, the softmax of 64 tokens) take longer
// than its bytes.
//
// A warp streams its blocks through a ring of its own in shared memory (bulk
// copies, one for the keys and one for the values of a block) and shares nothing
// with the others, so no barrier stands in its way.  The page numbers and scales
// of its next 32 blocks are looked up at once, a lane each.
//
// A piece is what a warp has of one tile (slot, key/value head, 8 rows).  A tile
// that lies in one warp's share is written out; of the others each warp leaves
// its part in the workspace, and another kernel (attention_join.cuh), launched while
// this one still runs, joins the parts in the list's order.

#include "attention_join.cuh"
#include "attention_ptx.cuh"

namespace qlin {
namespace attention {

__device__ unsigned int g_split_status = 0;

namespace {

constexpr int kThreads = kSplitWarps * 32;
constexpr int kRingBytes = 24576;             // of a warp: 6 chunks at D = 64, 3 at 128
constexpr int kInfo = 8;                      // blocks that the copies may run ahead
constexpr int kMaxSlots = 1024;
constexpr int kTailCost = 4;                  // of a tail, in blocks

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_split_status, bit); }

enum : unsigned { kCodes = 0, kTail = 1, kNone = 2 };

struct alignas(16) Info {  // of a block on its way
  float2 scales;  // of its keys and its values
  unsigned x;  // its place in the list
  unsigned kind;
};

struct Slot {  // blocks that the list has before it, its tokens with the new ones, its rows
  int list, total, row0, n;
};

template <int D>
struct Layout {
  static constexpr int kChunk = kBlock * D;          // bytes of a block's keys or values
  static constexpr int kRing = kRingBytes / kChunk;  // chunks in a warp's ring
  static constexpr int kInfoAt = kSplitWarps * kRingBytes;
  static constexpr int kBarAt = kInfoAt + kSplitWarps * kInfo * int(sizeof(Info));
  static constexpr int kScanAt = (kBarAt + kSplitWarps * kRing * 8 + 15) / 16 * 16;
  static constexpr int kListAt = kScanAt + kSplitWarps * 8;
  static int bytes(int slots) { return kListAt + slots * int(sizeof(Slot)); }
};

// Places of a slot in the list: its blocks, a tail counting for kTailCost of them
// (it is read without the ring, and takes about as long).
__device__ __forceinline__ unsigned places_of(int tokens) {
  return unsigned(tokens) / kBlock + (tokens % kBlock ? kTailCost : 0);
}

// The shares of `blocks` places: warp i has start(i) .. start(i + 1) - 1, the
// first `longer` warps one more than the others.
struct Shares {
  unsigned each, longer;
  __device__ Shares(unsigned blocks, unsigned warps)
      : each(blocks / warps), longer(blocks % warps) {}
  __device__ unsigned start(unsigned i) const { return i * each + min(i, longer); }
  __device__ unsigned of(unsigned x) const {
    const unsigned edge = longer * (each + 1);
    return x < edge ? x / (each + 1) : longer + (x - edge) / each;
  }
};

// A tile.
struct Piece {
  int slot, kvh, row0, here;    // here: rows of the tile
  unsigned first, last;         // the tile's blocks in the list
};

__device__ __forceinline__ Piece piece_at(const Slot* s_slot, int slots, int group, unsigned x) {
  int lo = 0, hi = slots;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (unsigned(s_slot[mid].list) <= x)
      lo = mid;
    else
      hi = mid;
  }
  const Slot sl = s_slot[lo];
  const int rows = sl.n * group;
  const unsigned n = places_of(sl.total), tile = (x - sl.list) / n;
  const unsigned row_tiles = unsigned(rows + kSplitTile - 1) / kSplitTile;
  Piece p;
  p.slot = lo;
  p.kvh = int(tile / row_tiles);
  p.row0 = int(tile % row_tiles) * kSplitTile;
  p.here = min(kSplitTile, rows - p.row0);
  p.first = sl.list + tile * n;
  p.last = p.first + n;
  return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    split_kernel(const Args a, float* parts, Split* splits) {
  using L = Layout<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + L::kScanAt);
  Slot* s_slot = reinterpret_cast<Slot*>(smem + L::kListAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kRingBytes;
  Info* info = reinterpret_cast<Info*>(smem + L::kInfoAt) + warp * kInfo;
  const uint32_t bar = ptx::smem_u32(smem + L::kBarAt) + warp * L::kRing * 8;
  if (lane == 0) {
    for (int i = 0; i < L::kRing; ++i) ptx::mbar_init(bar + 8 * i, 1);
    ptx::fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // the list: blocks before each slot
  int64_t all_blocks = 0;
  bool over = false;  // a slot has more rows than the call allows
  for (int b0 = 0; b0 < a.c.slots; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int64_t here = 0;
    SlotRows r = {0, 0, 0, false};
    if (b < a.c.slots) {
      r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
      if (blockIdx.x == 0) {
        if (r.bad) report(kStatusRows);
        if (r.n > a.max_new) report(kStatusMaxNew);
      }
      const int64_t rows = int64_t(r.n) * a.group;
      over |= r.n > a.max_new;
      if (rows <= kSplitRows && r.n <= a.max_new)
        here = (rows + kSplitTile - 1) / kSplitTile * a.c.kv_heads * places_of(r.held + r.n);
    }
    int64_t upto = here;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    int64_t before = all_blocks;
    for (int i = 0; i < kSplitWarps; ++i) {
      if (i < warp) before += s_scan[i];
      all_blocks += s_scan[i];
    }
    if (b < a.c.slots)
      s_slot[b] = Slot{int(before + upto - here), r.held + r.n, int(r.row0), r.n};
  }
  if (__syncthreads_or(over)) {  // such slots are left out: zeros
    for (int b = 0; b < a.c.slots; ++b) {
      const Slot sl = s_slot[b];
      if (sl.n <= a.max_new) continue;
      for (int row = blockIdx.x; row < sl.n; row += gridDim.x) {
        T* dst = static_cast<T*>(a.out) + int64_t(sl.row0 + row) * a.q_heads * D;
        for (int i = threadIdx.x * 8; i < a.q_heads * D; i += kThreads * 8)
          *reinterpret_cast<uint4*>(dst + i) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  // a CTA's warps are gridDim.x apart, so that a short list spreads over the CTAs
  const unsigned me = warp * gridDim.x + blockIdx.x;
  if (lane == 0) splits[me].last = -1;
  if (all_blocks > 0x3fffffff) {  // (more than a cache holds)
    if (threadIdx.x == 0) report(kStatusRows);
    return;
  }
  const unsigned blocks = unsigned(all_blocks);
  if (me >= blocks) return;
  const Shares shares(blocks, min(gridDim.x * kSplitWarps, blocks));
  const unsigned end = shares.start(me + 1);

  // ---- the copies
  unsigned next = shares.start(me);
  unsigned looked = next, known = next;  // lane l knows block looked + l < known
  bool keys_sent = false;                // the next block's keys are on the way
  unsigned sent = 0, used = 0;           // chunks
  unsigned begun = 0, done = 0;          // blocks
  const uint8_t* my_src = nullptr;
  float2 my_scales = make_float2(0.f, 0.f);
  unsigned my_kind = kNone;
  auto pump = [&] {
    while (next < end && sent - used < unsigned(L::kRing) && begun - done < unsigned(kInfo)) {
      if (next == known) {
        looked = next;
        known = min(next + 32, end);
        const unsigned x = next + lane;
        my_kind = kNone;
        if (x < known) {
          const Piece p = piece_at(s_slot, a.c.slots, a.group, x);
          const int j = int(x - p.first);
          const int full = s_slot[p.slot].total / kBlock;
          if (j == full) {
            my_kind = kTail;
          } else if (j < full) {
            const int64_t page = page_of(a.c, p.slot, j);
            if (page < 0) {
              report(kStatusPage);
            } else {
              const int64_t at = page * a.c.kv_heads + p.kvh;
              my_kind = kCodes;
              my_src = static_cast<const uint8_t*>(a.c.pages) + at * 2 * L::kChunk;
              my_scales = reinterpret_cast<const float2*>(a.c.scales)[at];
            }
          }
        }
      }
      const int from = int(next - looked);
      const bool codes = __shfl_sync(0xffffffffu, my_kind, from) == kCodes;
      if (lane == from) {
        if (!keys_sent) info[begun % kInfo] = Info{my_scales, next, my_kind};
        const unsigned slot = sent % L::kRing;
        if (codes)
          ptx::bulk_load(ptx::smem_u32(ring + slot * L::kChunk), my_src + (keys_sent ? L::kChunk : 0),
                    L::kChunk, bar + 8 * slot);
      }
      sent += codes;
      begun += !keys_sent;
      next += !codes || keys_sent;
      keys_sent = codes && !keys_sent;
    }
    __syncwarp();
  };

  Warp<T, D> w;
  Piece p = {};
  Split split = {-1, 0, 0, 0};
  unsigned x = 0, x_piece = 0;
  const T* qp = nullptr;
  int pos0 = 0, pos1 = 0, first_pos = 0;
  bool open = false;         // a piece is under way
  bool have_scores = false;  // of the block whose values come next
  float s[4][4];
  // A block takes two turns, its keys and its values, each of which gives a
  // chunk of the ring back; the copies go on in between.
  while (true) {
    pump();
    const bool through = done == begun;
    const Info f = info[done % kInfo];
    const bool same = open && !through && f.x < p.last;
    if (open && !same) {
      // ---- the piece is through: blocks x_piece .. x - 1 of the list
      open = false;
      float l[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] = w.l[i];
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
      }
      const Slot sl = s_slot[p.slot];
      if (x_piece == p.first && x == p.last) {
        const float f0 = share_of(l[0]), f1 = share_of(l[1]);
        const int row = p.row0 + g;
        T* dst = static_cast<T*>(a.out) +
                 (int64_t(sl.row0 + row / a.group) * a.q_heads + p.kvh * a.group +
                  row % a.group) * D + 2 * t;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t v =
                transpose8(pack2<T>(w.o[c][2 * h] * f0, w.o[c][2 * h + 1] * f1));
            if (g < p.here) *reinterpret_cast<uint32_t*>(dst + 16 * c + 8 * h) = v;
          }
      } else {
        float* part = parts + size_t(2 * me + (x_piece == p.first ? 1 : 0)) * kSplitPart<D>;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(part + (16 * c + 8 * h + g) * kSplitTile + 2 * t) =
                make_float2(w.o[c][2 * h], w.o[c][2 * h + 1]);
        if (g == 0) {
          *reinterpret_cast<float2*>(part + kSplitTile * D + 2 * t) = make_float2(w.m[0], w.m[1]);
          *reinterpret_cast<float2*>(part + kSplitTile * (D + 1) + 2 * t) = make_float2(l[0], l[1]);
        }
        if (x_piece == p.first)
          split = Split{int(shares.of(p.last - 1)), sl.row0, p.row0,
                        16 * p.kvh + p.here};
      }
    }
    if (through) break;
    if (!same) {
      // ---- a new piece
      open = true;
      x_piece = f.x;
      p = piece_at(s_slot, a.c.slots, a.group, f.x);
      const Slot sl = s_slot[p.slot];
      const int held = sl.total - sl.n, row = p.row0 + g;
      qp = g < p.here ? static_cast<const T*>(a.q) +
                            int64_t(sl.row0 + row / a.group) * a.q_stride +
                            (p.kvh * a.group + row % a.group) * D
                      : nullptr;
      // the two rows whose scores this lane holds
      pos0 = 2 * t < p.here ? held + (p.row0 + 2 * t) / a.group : -1;
      pos1 = 2 * t + 1 < p.here ? held + (p.row0 + 2 * t + 1) / a.group : -1;
      first_pos = held + p.row0 / a.group;
      w.load_q(qp, lane);
      w.init();
      w.prepare_q(a.scale_log2, lane);
    }
    x = f.x + 1;
    const int j = int(f.x - p.first);
    const int seen[2] = {pos0 - j * kBlock + 1, pos1 - j * kBlock + 1};
    if (f.kind == kCodes) {
      const unsigned slot = used % L::kRing;
      const uint8_t* chunk = ring + slot * L::kChunk;
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(bar + 8 * slot, (used / L::kRing) & 1))) {
        // the warp's other waits would run out one by one: it reports and goes, once the
        // copies under way have landed
        if (lane == 0) report(kStatusWait);
        for (; used < sent; ++used)
          ptx::mbar_wait(bar + 8 * (used % L::kRing), (used / L::kRing) & 1, 100000000ull);
        break;
      }
      if (!have_scores) {
        w.scores(chunk, s, lane);
      } else {
        uint32_t b[4][2];
        w.probabilities(s, b, f.scales.x, f.scales.y, seen, first_pos < j * kBlock + kBlock - 1,
                        lane);
        w.values(chunk, b, lane);
      }
      ++used;
      done += have_scores;
      have_scores = !have_scores;
    } else {
      if (f.kind == kTail)
        w.tail(static_cast<const T*>(a.c.tail) +
                   (int64_t(p.slot) * a.c.kv_heads + p.kvh) * 2 * kBlock * D,
               s_slot[p.slot].total - j * kBlock, qp, a.scale_log2, seen,
               first_pos + 1 - j * kBlock, lane);
      ++done;
    }
    ptx::fence_async_shared();
    __syncwarp();  // every lane has read the chunk and the info
  }
  if (lane == 0 && split.last >= 0) splits[me] = split;
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Args a, const SplitScratch sc) {
  grid_launch_dependents();
  grid_dependency_wait();
  join_split<T, D>(a, sc, blockIdx.x, gridDim.x);
}

template <typename T, int D>
cudaError_t launch_t(const Args& a, void* workspace, bool join, unsigned flags, cudaStream_t st) {
  using L = Layout<D>;
  static_assert(L::kListAt + kMaxSlots * int(sizeof(Slot)) <= 227 * 1024, "it fits");
  static std::atomic<unsigned long long> done{0};
  if (!allow_shared(reinterpret_cast<const void*>(split_kernel<T, D>), L::bytes(kMaxSlots), &done))
    return cudaGetLastError();
  const SplitScratch sc = split_scratch(workspace, sm_count());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sc.warps / kSplitWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(L::bytes(a.c.slots));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, split_kernel<T, D>, a, sc.parts, sc.splits);
  if (e != cudaSuccess || !join) return e;
  cfg.gridDim = dim3(unsigned(sm_count() * kSplitJoinPerSm));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D>, a, sc);
}

}  // namespace

size_t split_workspace_size(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  const size_t warps = size_t(split_scratch(nullptr, sm_count()).warps);
  return warps * (sizeof(Split) + 2 * kSplitTile * (head_dim + 2) * 4);
}

cudaError_t launch_split(const Args& a, void* workspace, bool join, unsigned flags,
                         cudaStream_t st) {
  if (a.c.dtype == QLIN_F16)
    return a.c.head_dim == 64 ? launch_t<__half, 64>(a, workspace, join, flags, st)
                              : launch_t<__half, 128>(a, workspace, join, flags, st);
  return a.c.head_dim == 64 ? launch_t<__nv_bfloat16, 64>(a, workspace, join, flags, st)
                            : launch_t<__nv_bfloat16, 128>(a, workspace, join, flags, st);
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
