// Attention of slots with many new rows (prompts and their chunks) on the
// tcgen05 tensor cores.
//
// A CTA takes 256 rows (new tokens times the query heads that share a key/value
// head) of one slot and key/value head, as two tiles of 128, and walks the
// blocks that they see.  Per block and tile
//   S [128 x 64] = q [128 x D] . keys^T      (q in shared memory)
//   P            = exp2(S * scale - max)     (row by row, in registers)
//   O [128 x D] += P [128 x 64] . values     (A: P in tensor memory, over S)
// with S, P and O in tensor memory and both operands of every product in f16:
// the codes are exact in it (a bf16 tail is scaled by a power of two for its keys and
// one for its values, exact down to 2^-28 and 2^-23 of the largest and rounded at 2^-31
// below; bf16 queries by one for each row, exact down to 2^-28).  S has two buffers a tile, so the
// scores of the next block are there when the exponentials of this one are done
// (with one, and q in tensor memory beside it, a tile waited for its products
// two fifths of the time: 375 us for two chunks of 2048 tokens over 6001).
//
//   warps 0..3, 4..7  a tile each, a thread for each row: the row's query to
//                     shared memory, then per block S from tensor memory,
//                     maximum, exponentials and sum (no other thread has a part
//                     of the row), P back; O is rescaled only when the maximum
//                     has grown by 2^8 (P stays within f16, and the last
//                     division makes up for it).
//   warps 8..11       widen the codes of keys and values to f16 in shared memory
//                     (128-byte swizzle, K-major), a ring of 3 blocks; the codes
//                     come through a ring of bulk copies.
//   warps 12, 13      issue the products of a tile each (one thread): one thread
//                     for both took 49 cycles for each 128 x 64 x 16 product,
//                     which the tensor core does in 32.
//
// Whole tiles leave some SMs idle in the last round.  What is left after the last
// full round (at most half of the SMs' number) is therefore cut along the cache,
// one piece for each SM; the pieces' sums go to the workspace, and the last kernel
// of the call joins them.
//
// What bounds it: at D = 128 a block of both tiles takes about 2650 cycles, and no
// unit is busy that long.  Its 32 products take 49 to 55 cycles each (1570 to 1760;
// the tensor core needs 32, but a product of the scores reads 6 KB of operands from
// shared memory, 48 cycles), all shared-memory traffic 192 KB (1536), the exponentials
// 1024; the last third is hand-overs between them.  bf16 spills 216 bytes there: 14
// warps leave 128 registers.  At D = 64 it is the way of a block through a tile's four
// warps (1660 cycles, of which the exponentials of both tiles take 1024; a quarter or
// an eighth of them by polynomial on the multiply-add pipe made it 10% longer).  Two
// chunks of 2048 over 6001, 32 query heads of 128: 351 us, 900 TFLOP/s; the products
// alone would be 163 us at the library's rate.

#include "attention_join.cuh"
#include "attention_ptx.cuh"

namespace qlin {
namespace attention {

__device__ unsigned int g_tile_status = 0;

namespace {

constexpr int kTileRows = 128;
constexpr int kTiles = 2;
constexpr int kCtaRows = kTiles * kTileRows;
constexpr int kSoftmaxWarps = 4 * kTiles;
constexpr int kWidenWarps = 4;
constexpr int kThreads = (kSoftmaxWarps + kWidenWarps + kTiles) * 32;
constexpr int kStages = 3;  // blocks of f16 operands
constexpr int kRaw = 4;     // blocks of codes
constexpr int kMaxCuts = 8;
constexpr float kSlack = 8.f;        // log2 of how far a row's maximum may lag

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_tile_status, bit); }

template <int D>
struct Layout {
  static constexpr int kKeys = 64 * D * 2;            // bytes of a block's f16 keys, or values
  static constexpr int kStage = 2 * kKeys;
  static constexpr int kCodes = 2 * 64 * D;           // a block's codes
  static constexpr int kQuery = kTileRows * D * 2;     // a tile's queries
  static constexpr int kQueryAt = kStages * kStage;
  static constexpr int kRawAt = kQueryAt + kTiles * kQuery;
  static constexpr int kBarAt = kRawAt + kRaw * kCodes;
  // barriers: operands full/empty, codes full; of a tile, for both buffers S full
  // and P's halves full, and q full, P used, O full
  static constexpr int kPerTile = 9;
  static constexpr int kBars = 2 * kStages + kRaw + kPerTile * kTiles;
  static constexpr int kScaleAt = kBarAt + kBars * 8;  // float2 of each stage
  static constexpr int kMiscAt = kScaleAt + kStages * 8;
  static constexpr int kBytes = kMiscAt + 64 + 1024;   // + alignment to 1024
  // tensor memory columns
  static constexpr int kS = 0;             // two buffers of 64 a tile (P over the first 32)
  static constexpr int kO = kTiles * 128;  // D a tile
  static_assert(kO + kTiles * D <= 512, "tensor memory");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void widen_barrier() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

// The work: pairs of tiles over all slots and key/value heads, the first `whole`
// as they are, the others in `cuts` pieces.
struct Plan {
  int pairs, whole, cuts;
};

__device__ __forceinline__ int64_t pairs_of(const Args& a, int b) {
  const SlotRows r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
  const int64_t rows = int64_t(r.n) * a.group;
  return rows > kSplitRows && r.n <= a.max_new
             ? (rows + kCtaRows - 1) / kCtaRows * a.c.kv_heads
             : 0;
}

// One warp; the same answer in every lane.
__device__ __forceinline__ Plan plan_of(const Args& a, int sms) {
  int64_t n = 0;
  for (int b = threadIdx.x & 31; b < a.c.slots; b += 32) n += pairs_of(a, b);
  for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  Plan p;
  p.pairs = int(n);
  const int rest = p.pairs % sms;
  p.cuts = rest ? min(sms / rest, kMaxCuts) : 1;
  p.whole = p.cuts > 1 ? p.pairs - rest : p.pairs;
  return p;
}

// A pair of tiles: the later ones of a slot, which see more, come first.
struct Work {
  SlotRows r;
  int slot, kvh, row0, n;  // n: blocks that its rows see
};
__device__ __forceinline__ Work work_at(const Args& a, int slot, int64_t place) {
  Work w;
  w.slot = slot;
  w.r = slot_rows(a.starts, a.c.lens, slot, a.n_tokens);
  const int rows = w.r.n * a.group, pairs = (rows + kCtaRows - 1) / kCtaRows;
  w.kvh = int(place % a.c.kv_heads);
  w.row0 = (pairs - 1 - int(place / a.c.kv_heads)) * kCtaRows;
  const int last = w.r.held + (min(w.row0 + kCtaRows, rows) - 1) / a.group;  // position seen
  w.n = last / kBlock + 1;
  return w;
}

// A piece's part in the workspace: sums [rows][D], then the rows' m and l.
template <int D>
constexpr int kPartFloats = kCtaRows * (D + 2);

// 16 codes -> 16 f16 values, 32 bytes
__device__ __forceinline__ void widen16(const uint4& w, uint4& lo, uint4& hi) {
  widen_codes(w.x, lo.x, lo.y);
  widen_codes(w.y, lo.z, lo.w);
  widen_codes(w.z, hi.x, hi.y);
  widen_codes(w.w, hi.z, hi.w);
}

// Byte offset of 16-byte chunk c of row r in a tile of 128-byte rows, swizzled.
__device__ __forceinline__ int swizzled(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const Args a, float* parts, int sms) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw_base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + L::kBarAt;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto raw_full = [&](int s) { return bars + 8u * (2 * kStages + s); };
  auto of_tile = [&](int t, int i) {
    return bars + 8u * (2 * kStages + kRaw + L::kPerTile * t + i);
  };
  auto s_full = [&](int t, int buf) { return of_tile(t, buf); };
  auto p_full = [&](int t, int buf, int half) { return of_tile(t, 2 + 2 * buf + half); };
  auto q_full = [&](int t) { return of_tile(t, 6); };
  auto p_used = [&](int t) { return of_tile(t, 7); };
  auto o_full = [&](int t) { return of_tile(t, 8); };
  float2* scales = reinterpret_cast<float2*>(smem + L::kScaleAt);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscAt);
  int* s_work = reinterpret_cast<int*>(smem + L::kMiscAt + 32);  // slot, place, cuts, cut
  float* s_top = reinterpret_cast<float*>(smem + L::kMiscAt + 8);  // of the four widening warps
  // the first of the tail's tokens with a value that is not finite, else kBlock
  int* s_lost = reinterpret_cast<int*>(smem + L::kMiscAt + 48);

  if (threadIdx.x == 0) {
    *s_lost = kBlock;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full(s), kWidenWarps);
      ptx::mbar_init(empty(s), kTiles);
    }
    for (int s = 0; s < kRaw; ++s) ptx::mbar_init(raw_full(s), 1);
    for (int t = 0; t < kTiles; ++t) {
      for (int i = 0; i < 2; ++i) {
        ptx::mbar_init(s_full(t, i), 1);
        for (int h = 0; h < 2; ++h) ptx::mbar_init(p_full(t, i, h), 4);
      }
      ptx::mbar_init(q_full(t), 4);
      ptx::mbar_init(p_used(t), 1);
      ptx::mbar_init(o_full(t), 1);
    }
    ptx::fence_mbar_init();
  }
  grid_dependency_wait();
  if (warp == 0) {
    const Plan plan = plan_of(a, sms);
    const int id = blockIdx.x;
    const int pair = id < plan.whole ? id : plan.whole + (id - plan.whole) / plan.cuts;
    int slot = -1;
    int64_t place = 0;
    const bool any = pair < plan.pairs && find_slot(a.c.slots, pair, &slot, &place,
                                                    [&](int b) { return pairs_of(a, b); });
    if (lane == 0) {
      s_work[0] = any ? slot : -1;
      s_work[1] = int(place);
      s_work[2] = id < plan.whole ? 1 : plan.cuts;
      s_work[3] = id < plan.whole ? 0 : (id - plan.whole) % plan.cuts;
    }
  }
  __syncthreads();
  const Work work = work_at(a, max(s_work[0], 0), s_work[1]);
  const int cuts = min(s_work[2], work.n), cut = s_work[3];
  if (s_work[0] < 0 || cut >= cuts) return;
  if (warp == kSoftmaxWarps + kWidenWarps) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (not before: a later kernel of the stream that takes tensor memory, and then waits
  // for this one, could stand on this SM first)
  grid_launch_dependents();

  const SlotRows r = work.r;
  const int b = work.slot, kvh = work.kvh, row0 = work.row0, rows = r.n * a.group;
  const int total = r.held + r.n;
  // this piece's blocks
  const int j0 = work.n * cut / cuts, n = work.n * (cut + 1) / cuts - j0;

  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ a row each
    const int tile = warp >> 2, quarter = warp & 3;
    const int row = row0 + tile * kTileRows + quarter * 32 + lane;
    const bool mine = row < rows;
    const int pos = mine ? r.held + row / a.group : 0x7fffffff;
    const uint32_t at = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t ts2 = at + L::kS + tile * 128, to = at + L::kO + tile * D;
    float factor = fabsf(a.scale_log2);
    {
      const T* src = static_cast<const T*>(a.q) +
                     (r.row0 + (mine ? row : 0) / a.group) * a.q_stride +
                     (kvh * a.group + (mine ? row : 0) % a.group) * D;
      uint32_t w[D / 2];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (mine) v = *reinterpret_cast<const uint4*>(src + 8 * i);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
      if (std::is_same<T, __nv_bfloat16>::value) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 2; ++i)
          top = fmaxf(top, fmaxf(fabsf(low_f32(w[i])), fabsf(high_f32(w[i]))));
        int e = int(__float_as_uint(top) >> 23) - 127 - 14;  // q * 2^-e is below 2^15
        e = max(-100, min(113, e));
        const float down = __uint_as_float(uint32_t(127 - e) << 23);
        factor *= __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < D / 2; ++i)
          w[i] = pack2<__half>(low_f32(w[i]) * down, high_f32(w[i]) * down);
      }
      // a negative scale goes to the query: the maximum is taken before scaling
      if (a.scale_log2 < 0.f) {
#pragma unroll
        for (int i = 0; i < D / 2; ++i) w[i] ^= 0x80008000u;
      }
      uint8_t* dst = smem + L::kQueryAt + tile * L::kQuery;
      const int here = quarter * 32 + lane;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<uint4*>(dst + i / 8 * (kTileRows * 128) + swizzled(here, i % 8)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      ptx::fence_async_shared();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_full(tile));
    }
    const int first = r.held + (row0 + tile * kTileRows) / a.group;  // of the tile: all see up to it
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int st = j % kStages, at_token = (j0 + j) * kBlock;
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(full(st), (j / kStages) & 1));
      if (!ok) break;
      // what goes by the scales alone, while the scores are computed
      const float2 ks = scales[st];
      // (never zero: a score of -infinity has to stay one)
      const float scale = ks.x < INFINITY ? fmaxf(factor * ks.x, 1e-30f) : INFINITY;
      // values that are not finite: the rows that see them are NaN, no other
      int lost = ks.y < INFINITY ? kBlock : 0;
      const float shift = lost ? weight_log2(ks.y) : 0.f;
      if (at_token + kBlock > total) lost = *s_lost;
      const int buf = j & 1;
      const uint32_t ts = ts2 + 64 * buf;
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full(tile, buf), (j >> 1) & 1));
      if (!ok) break;
      ptx::tc_fence_after();
      uint32_t v[64];
      ptx::tmem_ld_32x32b_x32(ts, *reinterpret_cast<uint32_t(*)[32]>(v));
      ptx::tmem_ld_32x32b_x32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
      ptx::tmem_wait_ld();
      if (first < at_token + kBlock - 1 || ks.x < 0.f) {
        // token i is seen where i <= seen (none of a block without a page)
        const int seen = ks.x < 0.f ? -1 : pos - at_token;
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i > seen) v[i] = 0xff800000u;  // -infinity
      }
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 64; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tops[e] = fmaxf(tops[e],
                          fmaxf(__uint_as_float(v[i + 2 * e]), __uint_as_float(v[i + 2 * e + 1])));
      const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale + shift;
      float keep = 1.f;
      if (top > m + kSlack || m == -INFINITY) {
        const float next = fmaxf(top, m);
        const float f = m == -INFINITY ? 1.f : exp2_fast(m - next);
        l *= f;
        keep = f;
        m = next;
      }
      if (j > 0 && __any_sync(0xffffffffu, keep != 1.f)) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(p_used(tile), (j - 1) & 1));
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          ptx::tmem_ld_32x32b_x16(to + c, o);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
          ptx::tmem_st_32x32b_x16(to + c, o);
        }
      }
      const float from = (m == -INFINITY ? 0.f : m) - shift;
      const float2 scale2 = make_float2(scale, scale), from2 = make_float2(-from, -from);
      float2 sum = make_float2(0.f, 0.f);
      // in halves of 32 tokens: the products on the first go on beside the second
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 x = make_float2(__uint_as_float(v[32 * h + 2 * i]),
                                 __uint_as_float(v[32 * h + 2 * i + 1]));
          x = __ffma2_rn(x, scale2, from2);
          x.x = exp2_fast(x.x);
          x.y = exp2_fast(x.y);
          sum = __fadd2_rn(sum, x);
          p[i] = pack2<__half>(x.x, x.y);
        }
        ptx::tmem_st_32x32b_x16(ts + 16 * h, p);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full(tile, buf, h));
      }
      l += (sum.x + sum.y) * exp2_fast(-shift);
      if (lost < kBlock && pos - at_token >= lost) l = NAN;
    }
    ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait(o_full(tile), 0));
    if (!ok) {
      if (lane == 0) report(kStatusWait);
    } else {
      ptx::tc_fence_after();
      const bool part = cuts > 1;
      const float f = share_of(l);
      T* dst = static_cast<T*>(a.out) +
               ((r.row0 + row / a.group) * a.q_heads + kvh * a.group + row % a.group) * D;
      float* sums = parts + size_t(blockIdx.x % sms) * kPartFloats<D>;
      const int here = tile * kTileRows + quarter * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        ptx::tmem_ld_32x32b_x32(to + c, o);
        ptx::tmem_wait_ld();
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(sums + here * D + c + 4 * i) =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack2<T>(__uint_as_float(o[8 * i + 2 * e]) * f,
                              __uint_as_float(o[8 * i + 2 * e + 1]) * f);
            *reinterpret_cast<uint4*>(dst + c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (part) {
        sums[kCtaRows * D + here] = m;
        sums[kCtaRows * (D + 1) + here] = l;
      }
    }
  } else if (warp < kSoftmaxWarps + kWidenWarps) {
    // ------------------------------------------------- codes to f16 operands
    const int i0 = (warp - kSoftmaxWarps) * 32 + lane;  // 0 .. 127
    const int full_blocks = min(n, total / kBlock - j0);  // of the piece's
    // thread 0 keeps the ring of codes filled; the pages of the next 32 blocks
    // are looked up at once, a lane each
    int sent = 0, looked = -32;
    int64_t my_page = -1;
    auto send = [&](int upto) {
      for (; sent < upto && sent < full_blocks; ++sent) {
        if (sent >= looked + 32) {
          looked = sent;
          my_page = sent + lane < full_blocks ? page_of(a.c, b, j0 + sent + lane) : -1;
        }
        const int64_t page = __shfl_sync(0xffffffffu, my_page, sent - looked);
        const int s = sent % kRaw;
        if (lane == 0) {
          if (page >= 0) {
            ptx::bulk_load(base + L::kRawAt + s * L::kCodes,
                           static_cast<const uint8_t*>(a.c.pages) +
                               (page * a.c.kv_heads + kvh) * L::kCodes,
                           L::kCodes, raw_full(s));
          } else {
            report(kStatusPage);
            ptx::mbar_arrive(raw_full(s));
          }
        }
      }
    };
    if (i0 < 32) send(kRaw);
    int looked2 = -32;
    float2 my_scales = make_float2(0.f, 0.f);
    bool my_good = false;
    bool ok = true;
    // (after a wait that gave up the warps go on without waiting: the others of
    // the warpgroup count on them at its barrier)
    for (int j = 0; j < n; ++j) {
      const int st = j % kStages;
      uint8_t* keys = smem + st * L::kStage;
      uint8_t* vals = keys + L::kKeys;
      if (j >= kStages && ok) ok = ptx::mbar_wait(empty(st), (j / kStages - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (j < full_blocks) {
        // scales of the next 32 blocks at once, a lane each
        if (j >= looked2 + 32) {
          looked2 = j;
          const int64_t page = j + lane < full_blocks ? page_of(a.c, b, j0 + j + lane) : -1;
          my_good = page >= 0;
          my_scales = my_good ? reinterpret_cast<const float2*>(
                                    a.c.scales)[page * a.c.kv_heads + kvh]
                              : make_float2(0.f, 0.f);
        }
        const float sx = __shfl_sync(0xffffffffu, my_scales.x, j - looked2);
        const float sy = __shfl_sync(0xffffffffu, my_scales.y, j - looked2);
        const bool good = __shfl_sync(0xffffffffu, int(my_good), j - looked2);
        if (i0 == 0) scales[st] = make_float2(good ? sx : -1.f, sy);
        const int s = j % kRaw;
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(raw_full(s), (j / kRaw) & 1));
        const uint8_t* raw = smem + L::kRawAt + s * L::kCodes;
        constexpr int kUnits = D / 16;  // of 16 codes in a key row
#pragma unroll
        for (int k = 0; k < 64 * kUnits / 128; ++k) {
          const int u = k * 128 + i0, tok = u / kUnits, c = u % kUnits;
          uint4 lo, hi;
          uint4 w = *reinterpret_cast<const uint4*>(raw + 16 * u);
          if (!good) w = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
          widen16(w, lo, hi);
          uint8_t* dst = keys + (c / 4) * 8192;
          *reinterpret_cast<uint4*>(dst + swizzled(tok, 2 * (c % 4))) = lo;
          *reinterpret_cast<uint4*>(dst + swizzled(tok, 2 * (c % 4) + 1)) = hi;
        }
#pragma unroll
        for (int k = 0; k < D * 4 / 128; ++k) {
          const int u = k * 128 + i0, d = u / 4, c = u % 4;
          uint4 lo, hi;
          uint4 w = *reinterpret_cast<const uint4*>(raw + 64 * D + 16 * u);
          if (!good) w = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
          widen16(w, lo, hi);
          *reinterpret_cast<uint4*>(vals + swizzled(d, 2 * c)) = lo;
          *reinterpret_cast<uint4*>(vals + swizzled(d, 2 * c + 1)) = hi;
        }
      } else {
        // the tail: T as it is (f16), or scaled by a power of two (bf16); what
        // lies beyond its last token is undefined and becomes zero, as do values
        // that are not finite (0 times them would be NaN in the rows that do not see
        // their token)
        const T* src = static_cast<const T*>(a.c.tail) +
                       (int64_t(b) * a.c.kv_heads + kvh) * 2 * kBlock * D;
        const int count = total - (j0 + j) * kBlock;
        float2 sc = make_float2(1.f, 1.f);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const T* from = src + half * kBlock * D;
          float down = 1.f;
          if (std::is_same<T, __nv_bfloat16>::value) {
            float top = 0.f;
#pragma unroll 1
            for (int u = i0; u < kBlock * D; u += 128) {
              const int tok = half ? u % kBlock : u / D;
              const float v = fabsf(Act<T>::to_f32(from[u]));
              if (tok < count && v < INFINITY) top = fmaxf(top, v);
            }
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            widen_barrier();
            if (lane == 0) s_top[warp - kSoftmaxWarps] = top;
            widen_barrier();
            top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
            // keys to below 2^15; values to below 2^7, as codes are, for a weight like theirs
            int e = int(__float_as_uint(top) >> 23) - 127 - (half ? 6 : 14);
            e = max(-100, min(121, e));
            down = __uint_as_float(uint32_t(127 - e) << 23);
            (half ? sc.y : sc.x) = __uint_as_float(uint32_t(127 + e) << 23);
          }
#pragma unroll 1
          for (int u = i0; u < kBlock * D / 8; u += 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(from + 8 * u);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
            uint32_t y[4];
            const int tok = half ? 8 * u % kBlock : 8 * u / D;  // (values: the first of eight)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t v = x[e];
              if (std::is_same<T, __nv_bfloat16>::value)
                v = pack2<__half>(low_f32(v) * down, high_f32(v) * down);
              const int t0 = half ? tok + 2 * e : tok, t1 = half ? t0 + 1 : tok;
              uint32_t lo = t0 < count ? v & 0xffffu : 0u, hi = t1 < count ? v & 0xffff0000u : 0u;
              if (half && (lo & 0x7c00u) == 0x7c00u) {
                atomicMin(s_lost, t0);
                lo = 0;
              }
              if (half && (hi & 0x7c000000u) == 0x7c000000u) {
                atomicMin(s_lost, t1);
                hi = 0;
              }
              y[e] = lo | hi;
            }
            const int at = half ? swizzled(8 * u / kBlock, 8 * u % kBlock / 8)
                                : (8 * u % D) / 64 * 8192 + swizzled(tok, 8 * u % 64 / 8);
            *reinterpret_cast<uint4*>((half ? vals : keys) + at) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        if (i0 == 0) scales[st] = sc;
      }
      ptx::fence_async_shared();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full(st));
      // the codes are read: the slot takes the next block.  The ring's barrier
      // orders the four warps' reads before the copy.
      widen_barrier();
      if (i0 < 32 && ok) send(j + 1 + kRaw);
    }
    if (!ok) {
      if (lane == 0) report(kStatusWait);
      if (i0 == 0)  // copies under way land before the CTA goes
        for (int k = max(0, sent - kRaw); k < sent; ++k)
          ptx::mbar_wait(raw_full(k % kRaw), (k / kRaw) & 1, 100000000ull);
    }
  } else if (lane == 0) {
    // ------------------------------------------------ the products of a tile
    constexpr uint32_t id_s = ptx::idesc_f16(0, kTileRows, kBlock);
    constexpr uint32_t id_o = ptx::idesc_f16(0, kTileRows, D);
    const int t = warp - kSoftmaxWarps - kWidenWarps;
    const uint32_t ts2 = tmem + L::kS + t * 128, to = tmem + L::kO + t * D;
    const uint64_t q_desc = ptx::sw128_kmajor_desc(base + L::kQueryAt + t * L::kQuery);
    // the scores of block j, into its buffer
    auto scores = [&](int j) {
      const uint64_t k_desc = ptx::sw128_kmajor_desc(base + j % kStages * L::kStage);
#pragma unroll
      for (int p = 0; p < D / 64; ++p)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::mma_f16_ss(ts2 + 64 * (j & 1), q_desc + (p * (kTileRows * 128) >> 4) + 2 * k,
                          k_desc + (p * 8192 >> 4) + 2 * k, id_s, p + k > 0);
      ptx::mma_commit(s_full(t, j & 1));
    };
    bool ok = ptx::mbar_wait(q_full(t), 0);
    for (int j = 0; j < 2 && j < n && ok; ++j) {
      ok = ptx::mbar_wait(full(j), 0);
      ptx::tc_fence_after();
      if (ok) scores(j);
    }
    for (int j = 0; j < n && ok; ++j) {
      const int st = j % kStages;
      const uint32_t ts = ts2 + 64 * (j & 1);
      const uint64_t desc = ptx::sw128_kmajor_desc(base + st * L::kStage + L::kKeys);
      for (int h = 0; h < 2 && ok; ++h) {
        ok = ptx::mbar_wait(p_full(t, j & 1, h), (j >> 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 2; ++k)
          ptx::mma_f16_ts(to, ts + 16 * h + 8 * k, desc + 4 * h + 2 * k, id_o, j + h + k > 0);
      }
      if (!ok) break;
      ptx::mma_commit(empty(st));
      ptx::mma_commit(p_used(t));
      if (j + 2 < n) {  // (its buffer is free: products run in the order of their issue)
        ok = ptx::mbar_wait(full((j + 2) % kStages), ((j + 2) / kStages) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        scores(j + 2);
      }
    }
    ptx::mma_commit(o_full(t));
    // every product has to be through before tensor memory is given back
    if (!ptx::mbar_wait(o_full(t), 0) || !ok) report(kStatusWait);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + kWidenWarps) ptx::tmem_dealloc(tmem, 512);
}

// Joins the pieces, a warp for each row.  The CTA is `block` of `blocks`.
template <typename T, int D>
__device__ void join_pieces(const Args& a, const float* parts, int sms, int block, int blocks) {
  constexpr int kWarps = kJoinThreads / 32;
  const int lane = threadIdx.x & 31, warp = block * kWarps + (threadIdx.x >> 5);
  const Plan plan = plan_of(a, sms);
  if (plan.cuts == 1) return;
  for (int64_t i = warp; i < int64_t(plan.pairs - plan.whole) * kCtaRows; i += blocks * kWarps) {
    const int at = int(i / kCtaRows), row = int(i % kCtaRows);
    int slot = 0;
    int64_t place = 0;
    if (!find_slot(a.c.slots, plan.whole + at, &slot, &place,
                   [&](int b) { return pairs_of(a, b); }))
      return;
    const Work w = work_at(a, slot, place);
    if (w.row0 + row >= w.r.n * a.group) continue;
    const int cuts = min(plan.cuts, w.n);
    if (cuts == 1) continue;  // (written out)
    float m[kMaxCuts], l[kMaxCuts], top = -INFINITY, sum = 0.f;
    float o[D / 32] = {};
    const float* first = parts;
    auto part = [&](int k) {
      return first + size_t((plan.whole + at * plan.cuts + k) % sms) * kPartFloats<D>;
    };
#pragma unroll
    for (int k = 0; k < kMaxCuts; ++k) {
      m[k] = k < cuts ? __ldcg(part(k) + kCtaRows * D + row) : -INFINITY;
      l[k] = k < cuts ? __ldcg(part(k) + kCtaRows * (D + 1) + row) : 0.f;
      top = fmaxf(top, m[k]);
    }
#pragma unroll
    for (int k = 0; k < kMaxCuts; ++k) {
      if (l[k] == 0.f) continue;  // (no such piece, or none of its blocks is seen)
      const float f = m[k] == -INFINITY ? 0.f : exp2_fast(m[k] - top);
      sum += l[k] * f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] += __ldcg(part(k) + row * D + 32 * e + lane) * f;
    }
    const int rr = w.row0 + row;
    T* dst = static_cast<T*>(a.out) +
             ((w.r.row0 + rr / a.group) * a.q_heads + w.kvh * a.group + rr % a.group) * D;
    const float f = share_of(sum);
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
      dst[32 * e + lane] = Act<T>::from_f32_rn(o[e] * f);
  }
}

// After both kernels, what both left: the pieces by the first kTileJoinPerSm * sms
// CTAs, the split kernel's parts by the others.
constexpr int kTileJoinPerSm = 1;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const Args a, const float* parts, const SplitScratch sc, int sms) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int pieces = kTileJoinPerSm * sms;
  if (int(blockIdx.x) < pieces)
    join_pieces<T, D>(a, parts, sms, blockIdx.x, pieces);
  else
    join_split<T, D>(a, sc, blockIdx.x - pieces, gridDim.x - pieces);
}

template <typename T, int D>
cudaError_t launch_t(const Args& a, void* workspace, const SplitScratch& sc, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  if (!allow_shared(reinterpret_cast<const void*>(tile_kernel<T, D>), Layout<D>::kBytes, &done))
    return cudaGetLastError();
  const int sms = sm_count();
  float* parts = static_cast<float*>(workspace);
  cudaLaunchConfig_t cfg = {};
  // pairs of tiles of all slots, and the pieces of the last round
  const int64_t most = (a.n_tokens * a.group / kCtaRows + a.c.slots) * a.c.kv_heads + sms;
  cfg.gridDim = dim3(unsigned(most));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<D>::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tile_kernel<T, D>, a, parts, sms);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(unsigned((kTileJoinPerSm + kSplitJoinPerSm) * sms));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D>, a, static_cast<const float*>(parts), sc, sms);
}

}  // namespace

size_t tile_workspace_size(int head_dim) {
  return head_dim == 64 || head_dim == 128 ? size_t(sm_count()) * kCtaRows * (head_dim + 2) * 4 : 0;
}

cudaError_t launch_tile(const Args& a, void* workspace, void* split_workspace, cudaStream_t st) {
  const SplitScratch sc = split_scratch(split_workspace, sm_count());
  if (a.c.dtype == QLIN_F16)
    return a.c.head_dim == 64 ? launch_t<__half, 64>(a, workspace, sc, st)
                              : launch_t<__half, 128>(a, workspace, sc, st);
  return a.c.head_dim == 64 ? launch_t<__nv_bfloat16, 64>(a, workspace, sc, st)
                            : launch_t<__nv_bfloat16, 128>(a, workspace, sc, st);
}

cudaError_t tile_take_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tile_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_tile_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace attention
}  // namespace qlin
