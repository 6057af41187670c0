// Rotary positions and the append to the 8-bit key/value cache (qlin.h has the
// formats), the table of cosines and sines, and the cache's reconstruction.
//
// One launch does two kinds of work:
//   token warps   four warps per new token: they turn its queries and, where
//                 the token's block stays incomplete, its keys, which go with
//                 its values to the slot's tail;
//   block CTAs    one CTA per block that the call completes and key/value
//                 head: gathers the block's 64 tokens (the tail's, then new
//                 ones), takes the largest magnitude of the keys and of the
//                 values, and writes the codes.
// The tail has room for one block: where a slot completes a block with tokens
// from the tail and also starts a new one, the first block's CTA writes the
// new tail, after it has read the old.
//
// It moves 2 bytes in and 2 (queries) or 1 (blocks) out per element and does a
// handful of operations on each: memory bounds long prompts, launch and
// latency a decode step.  4 prompts of 2048 tokens, 32 + 8 + 8 heads of 128, take
// 45 us (at 49, their token warps alone took 42, their block CTAs 31); both wait
// for loads, with all of an SM's threads in flight.  32 decoded tokens take 7.2 us,
// 4.8 in a graph.
// Angles come from a table made in 64 bits: at
// position 100000 a float32 angle would be off by up to 4e-3 radians.

#include <cmath>
#include <type_traits>

#include "kv_cache.cuh"

namespace qlin {

__device__ unsigned int g_rope_status = 0;

namespace {

// Threads of a CTA: one for each 16 elements of a block's keys.  (256 at both head
// dimensions left a thread at 128 with twice the registers, and an SM with half the
// loads in flight: 59 us for 4 prompts of 2048.)
template <int D>
constexpr int kThreads = kBlock * (D / 16);

// Warps that share a token: the heads of one warp come two after two.  (1, 2, 4
// and 8: 32 decoded tokens in 19, 15, 15 and 15 us, 4 prompts of 2048 in 74, 66,
// 62 and 68.)
constexpr int kParts = 4;

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_rope_status, bit); }

// Eight elements as four pairs, the first of a pair in the low half.
struct Vec8 {
  uint32_t w[4];
};
template <typename T>
__device__ __forceinline__ Vec8 load8(const T* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return Vec8{{v.x, v.y, v.z, v.w}};
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec8& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  using T2 = typename Act<T>::T2;
  const T2 v = *reinterpret_cast<const T2*>(&w);
  return make_float2(Act<T>::to_f32(v.x), Act<T>::to_f32(v.y));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float2 v) {
  typename Act<T>::T2 r;
  r.x = Act<T>::from_f32_rn(v.x);
  r.y = Act<T>::from_f32_rn(v.y);
  return *reinterpret_cast<uint32_t*>(&r);
}

// A unit is 16 elements of a head, as two runs of 8 that pair up: units below
// rot/16 turn (half layout: 8u.. with rot/2 + 8u..; interleaved: 16u..), the
// others only move.
struct Unit {
  int at0, at1;  // first element of each run
};
__device__ __forceinline__ Unit unit_of(int u, int rot, bool interleaved) {
  const bool split = !interleaved && 16 * u < rot;
  return split ? Unit{8 * u, rot / 2 + 8 * u} : Unit{16 * u, 16 * u + 8};
}

// Products and their difference are rounded one by one, as the definition's
// float32 operations are: a fused multiply-add would round differently and
// could change a code.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float na = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float nb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = na;
  b = nb;
}

// A unit's 8 cosines and sines, from the position's row of the table.
struct Angles {
  float4 v[4];
};
__device__ __forceinline__ Angles angles_of(const float* row, int u, int rot) {
  Angles t;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    t.v[i] = 16 * u < rot ? reinterpret_cast<const float4*>(row + 16 * u)[i]
                          : make_float4(1.f, 0.f, 1.f, 0.f);
  return t;
}

template <typename T>
__device__ __forceinline__ void rotate_unit(Vec8& x, Vec8& y, int u, int rot, bool interleaved,
                                            const Angles& angles) {
  if (16 * u >= rot) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 a = unpack<T>(x.w[i]), b = unpack<T>(y.w[i]);
    if (interleaved) {
      const float4 t = angles.v[i / 2], z = angles.v[2 + i / 2];
      turn(a.x, a.y, i % 2 ? t.z : t.x, i % 2 ? t.w : t.y);
      turn(b.x, b.y, i % 2 ? z.z : z.x, i % 2 ? z.w : z.y);
    } else {
      const float4 t = angles.v[i];
      turn(a.x, b.x, t.x, t.y);
      turn(a.y, b.y, t.z, t.w);
    }
    x.w[i] = pack<T>(a);
    y.w[i] = pack<T>(b);
  }
}

// The code of v in a block of this scale; 128 throughout where the scale is 0, or
// infinite (an element was not finite: the block stands for 0 times infinity, NaN).
__device__ __forceinline__ unsigned code_of(float v, float scale) {
  if (!(scale > 0.f && scale < INFINITY)) return 128u;
  return unsigned(fminf(fmaxf(rintf(__fdiv_rn(v, scale)), -127.f), 127.f) + 128.f);
}

template <typename T>
__device__ __forceinline__ uint2 codes_of(const Vec8& v, float scale) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack<T>(v.w[2 * i]), b = unpack<T>(v.w[2 * i + 1]);
    r[i] = code_of(a.x, scale) | code_of(a.y, scale) << 8 | code_of(b.x, scale) << 16 |
           code_of(b.y, scale) << 24;
  }
  return make_uint2(r[0], r[1]);
}

// The largest magnitude, as bits: they order as the magnitudes do, with infinity above
// all numbers and NaN above that, where fmaxf would drop it.
template <typename T>
__device__ __forceinline__ uint32_t largest(const Vec8& v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack<T>(v.w[i]);
    top = max(top, max(__float_as_uint(fabsf(a.x)), __float_as_uint(fabsf(a.y))));
  }
  return top;
}

// 16 elements to a column.
template <typename T>
__device__ __forceinline__ void column_to(T* to, int stride, const Vec8& a, const Vec8& b) {
  uint16_t* p = reinterpret_cast<uint16_t*>(to);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint32_t w = (e < 8 ? a : b).w[e % 8 / 2];
    p[e * stride] = uint16_t(e % 2 ? w >> 16 : w);
  }
}

template <int WARPS>
__device__ __forceinline__ float block_max(uint32_t v, uint32_t* partial) {
  for (int d = 16; d; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = v;
  __syncthreads();
  v = partial[0];
  for (int i = 1; i < WARPS; ++i) v = max(v, partial[i]);
  return __uint_as_float(min(v, 0x7f800000u));  // (infinity for NaN)
}

struct Args {
  const void* qkv;
  int64_t qkv_stride;
  void* q_out;
  const float* table;
  int64_t n_positions;
  int rot, interleaved;
  qlin_kv_cache c;
  const int32_t* starts;
  int64_t n_tokens;
  int q_heads;
  int64_t block_items;  // room for completed blocks, over all slots
};

// Whether all of a slot's rows can be taken: its blocks fit and its positions
// are in the table.
__device__ __forceinline__ bool slot_fits(const Args& a, const SlotRows& r) {
  const int64_t total = int64_t(r.held) + r.n;
  return !r.bad && total / kBlock <= a.c.max_blocks && (a.rot == 0 || total <= a.n_positions);
}

// A share of one new token's heads: the queries, and keys and values to the tail
// where that is this warp's to write.  A lane's units differ by the head alone, so
// it looks its angles up once.
template <typename T, int D>
__device__ void token_warp(const Args& a, int64_t t, int part) {
  constexpr int kUnits = D / 16, kHeads = 32 / kUnits;  // of a head; heads at a time
  const int lane = threadIdx.x & 31;
  int b = -1;  // the token's slot
  for (int s0 = 0; s0 < a.c.slots; s0 += 32) {
    const int s = s0 + lane;
    const bool mine = s < a.c.slots && a.starts[s] <= t && t < a.starts[s + 1];
    const unsigned found = __ballot_sync(0xffffffffu, mine);
    if (found) {
      b = s0 + __ffs(found) - 1;
      break;
    }
  }
  if (b < 0) return;  // a row that no slot owns
  const SlotRows r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
  if (!slot_fits(a, r)) {
    if (lane == 0)
      report(r.bad ? kStatusRows
                   : (int64_t(r.held) + r.n) / kBlock > a.c.max_blocks ? kStatusPage
                                                                       : kStatusPosition);
    return;
  }
  const int pos = r.held + int(t - r.row0), u = lane % kUnits;
  const T* row = static_cast<const T*>(a.qkv) + t * a.qkv_stride;
  const Angles angles = angles_of(a.table + int64_t(pos) * a.rot, u, a.rot);
  const Unit un = unit_of(u, a.rot, a.interleaved);
  T* out = static_cast<T*>(a.q_out) + t * a.q_heads * D;
  const int q1 = a.q_heads * (part + 1) / kParts;
  // two heads' loads before the first store (which could be to the same memory,
  // for all that the compiler knows)
  for (int h = a.q_heads * part / kParts + lane / kUnits; h < q1; h += 2 * kHeads) {
    const bool two = h + kHeads < q1;
    const T* from = row + h * D;
    T* to = out + h * D;
    Vec8 x0 = load8(from + un.at0), y0 = load8(from + un.at1), x1 = x0, y1 = y0;
    if (two) {
      x1 = load8(from + kHeads * D + un.at0);
      y1 = load8(from + kHeads * D + un.at1);
    }
    rotate_unit<T>(x0, y0, u, a.rot, a.interleaved, angles);
    store8(to + un.at0, x0);
    store8(to + un.at1, y0);
    if (two) {
      rotate_unit<T>(x1, y1, u, a.rot, a.interleaved, angles);
      store8(to + kHeads * D + un.at0, x1);
      store8(to + kHeads * D + un.at1, y1);
    }
  }
  const int total = r.held + r.n;
  const bool stays = pos / kBlock == total / kBlock;
  const bool left_to_block = total / kBlock > r.held / kBlock && r.held % kBlock;
  if (!stays || left_to_block) return;
  const int at = pos % kBlock, k1 = a.c.kv_heads * (part + 1) / kParts;
  for (int h = a.c.kv_heads * part / kParts + lane / kUnits; h < k1; h += kHeads) {
    T* tail = static_cast<T*>(a.c.tail) + (int64_t(b) * a.c.kv_heads + h) * 2 * kBlock * D;
    const T* k = row + (a.q_heads + h) * D;
    const T* v = row + (a.q_heads + a.c.kv_heads + h) * D + 16 * u;
    Vec8 x = load8(k + un.at0), y = load8(k + un.at1);
    const Vec8 v0 = load8(v), v1 = load8(v + 8);
    rotate_unit<T>(x, y, u, a.rot, a.interleaved, angles);
    store8(tail + at * D + un.at0, x);
    store8(tail + at * D + un.at1, y);
    column_to(tail + kBlock * D + 16 * u * kBlock + at, kBlock, v0, v1);
  }
}

template <typename T, int D>
__device__ void block_cta(const Args& a, int64_t item, int h) {
  constexpr int kWarps = kThreads<D> / 32;
  constexpr int kStride = kBlock + 2;  // of a staged value row: spreads the banks
  __shared__ alignas(16) T staged[D * kStride];
  __shared__ uint32_t partial[kWarps];
  __shared__ int s_slot, s_place;
  __shared__ int64_t s_page;
  __shared__ SlotRows s_rows;
  if (threadIdx.x < 32) {
    int b = -1;
    int64_t place = 0;
    const bool any = find_slot(a.c.slots, item, &b, &place, [&](int s) -> int64_t {
      const SlotRows r = slot_rows(a.starts, a.c.lens, s, a.n_tokens);
      return slot_fits(a, r) ? (int64_t(r.held) + r.n) / kBlock - r.held / kBlock : 0;
    });
    if (threadIdx.x == 0) {
      s_slot = any ? b : -1;
      if (any) {
        s_rows = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
        s_place = int(place);
        s_page = page_of(a.c, b, s_rows.held / kBlock + int(place));
      }
    }
  }
  __syncthreads();
  const int b = s_slot;
  if (b < 0) return;
  const SlotRows r = s_rows;
  const int j = r.held / kBlock + s_place;
  const int old = j == r.held / kBlock ? r.held % kBlock : 0;  // tokens that the tail holds
  const int64_t page = s_page;
  if (page < 0 && threadIdx.x == 0) report(kStatusPage);
  T* tail = static_cast<T*>(a.c.tail) + (int64_t(b) * a.c.kv_heads + h) * 2 * kBlock * D;
  // rows of the block's new tokens: token i of the block is row first + i
  const int64_t first = r.row0 + int64_t(j) * kBlock - r.held;
  const T* qkv = static_cast<const T*>(a.qkv);

  // keys: a unit a thread
  const int tok = threadIdx.x / (D / 16), u = threadIdx.x % (D / 16);
  const Unit un = unit_of(u, a.rot, a.interleaved);
  const T* k = tok < old ? tail + tok * D
                         : qkv + (first + tok) * a.qkv_stride + (a.q_heads + h) * D;
  // all loads first: new values (transposed on their way through shared memory: a
  // warp's lanes are tokens, so that its stores run along a row), and the tail's,
  // which stand transposed already: dimension d, tokens t0 ..
  const int wi = threadIdx.x >> 5, vu = wi % (D / 16);
  const int vtok = wi / (D / 16) * 32 + (threadIdx.x & 31);
  const int d = threadIdx.x / 4, t0 = (threadIdx.x % 4) * 16;
  Vec8 kx = load8(k + un.at0), ky = load8(k + un.at1), nv[2], vv[2];
  const Angles angles =
      angles_of(a.table + (int64_t(j) * kBlock + tok) * a.rot, u, tok < old ? 0 : a.rot);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (vtok >= old)
      nv[p] = load8(qkv + (first + vtok) * a.qkv_stride + (a.q_heads + a.c.kv_heads + h) * D +
                    16 * vu + 8 * p);
    if (t0 + 8 * p < old) vv[p] = load8(tail + kBlock * D + d * kBlock + t0 + 8 * p);
  }
  if (vtok >= old) column_to(staged + 16 * vu * kStride + vtok, kStride, nv[0], nv[1]);
  if (tok >= old) rotate_unit<T>(kx, ky, u, a.rot, a.interleaved, angles);
  uint32_t top = max(largest<T>(kx), largest<T>(ky));
  // (the barriers of block_max order `staged` too)
  const float k_scale = __fdiv_rn(block_max<kWarps>(top, partial), 127.f);
  const uint32_t* from = reinterpret_cast<const uint32_t*>(staged + d * kStride + t0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t& w = vv[i / 4].w[i % 4];
    const int at = t0 + 2 * i;  // of the pair's first token
    if (at >= old)
      w = from[i];
    else if (at + 1 >= old)
      w = (w & 0xffffu) | (from[i] & 0xffff0000u);
  }
  top = max(largest<T>(vv[0]), largest<T>(vv[1]));
  const float v_scale = __fdiv_rn(block_max<kWarps>(top, partial), 127.f);
  if (page >= 0) {
    uint8_t* codes = static_cast<uint8_t*>(a.c.pages) + (page * a.c.kv_heads + h) * 2 * kBlock * D;
    if (threadIdx.x == 0) {
      float* s = a.c.scales + (page * a.c.kv_heads + h) * 2;
      s[0] = k_scale;
      s[1] = v_scale;
    }
    *reinterpret_cast<uint2*>(codes + tok * D + un.at0) = codes_of<T>(kx, k_scale);
    *reinterpret_cast<uint2*>(codes + tok * D + un.at1) = codes_of<T>(ky, k_scale);
    const uint2 lo = codes_of<T>(vv[0], v_scale), hi = codes_of<T>(vv[1], v_scale);
    *reinterpret_cast<uint4*>(codes + kBlock * D + d * kBlock + t0) =
        make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  // the new tail, where the old one had tokens of this block (all read above:
  // the barriers of block_max lie in between)
  const int total = r.held + r.n, pos = total / kBlock * kBlock + tok;
  if (old && pos < total) {
    const T* row = qkv + (r.row0 + pos - r.held) * a.qkv_stride;
    const T* nk = row + (a.q_heads + h) * D;
    const T* next = row + (a.q_heads + a.c.kv_heads + h) * D + 16 * u;
    Vec8 x = load8(nk + un.at0), y = load8(nk + un.at1);
    const Vec8 v0 = load8(next), v1 = load8(next + 8);
    rotate_unit<T>(x, y, u, a.rot, a.interleaved,
                   angles_of(a.table + int64_t(pos) * a.rot, u, a.rot));
    store8(tail + tok * D + un.at0, x);
    store8(tail + tok * D + un.at1, y);
    column_to(tail + kBlock * D + 16 * u * kBlock + tok, kBlock, v0, v1);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads<D>, 1024 / kThreads<D>) rope_append_kernel(const Args a) {
  constexpr int kWarps = kThreads<D> / 32;
  grid_launch_dependents();
  grid_dependency_wait();
  // block CTAs first: they take longer
  const int64_t blocks = a.block_items * a.c.kv_heads;
  if (blockIdx.x < blocks) {
    block_cta<T, D>(a, blockIdx.x / a.c.kv_heads, blockIdx.x % a.c.kv_heads);
  } else {
    const int64_t i = (blockIdx.x - blocks) * kWarps + (threadIdx.x >> 5), t = i / kParts;
    if (t < a.n_tokens) token_warp<T, D>(a, t, int(i % kParts));
  }
}

// ------------------------------------------------------------------ the table
__global__ void rope_table_kernel(float* table, int64_t n, int pairs, double base, double factor,
                                  double short_w, double long_w) {
  const double two_pi = 6.283185307179586476925286766559;
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n * pairs) return;
  const int64_t pos = i / pairs;
  const int p = int(i % pairs);
  double f = pow(base, -double(p) / pairs);
  const double wave = two_pi / f;
  if (factor > 1.0 && wave > short_w) {
    double keep = 0.0;  // share of the unscaled frequency
    if (long_w > short_w && wave < long_w)
      keep = short_w > 0.0 ? (1.0 / wave - 1.0 / long_w) / (1.0 / short_w - 1.0 / long_w) : 0.0;
    f = keep * f + (1.0 - keep) * f / factor;
  }
  double s, c;
  sincos(double(pos) * f, &s, &c);
  reinterpret_cast<float2*>(table)[i] = make_float2(float(c), float(s));
}

// --------------------------------------------------------------- reconstruction
// 8192 codes of a page a CTA (a page has a multiple of them), eight at a time a thread,
// so that a warp's stores run on without gaps: 103 pages of 8 heads of 128 (13.5 MB to
// 27) in 8.6 us (16 at a time, in two stores apart: 10.3).
constexpr int kDequantThreads = 256, kDequantCodes = 8192;

template <typename T>
__global__ void __launch_bounds__(kDequantThreads)
    cache_dequant_kernel(const qlin_kv_cache c, const int32_t* __restrict__ ids, T* out) {
  constexpr int kTurns = kDequantCodes / (8 * kDequantThreads);
  const int64_t per_page = int64_t(c.kv_heads) * 2 * kBlock * c.head_dim;
  const int64_t page = ids[blockIdx.y];
  const bool good = page >= 0 && page < c.n_pages;
  if (!good && blockIdx.x == 0 && threadIdx.x == 0) report(kStatusPage);
  const int64_t at = int64_t(blockIdx.x) * kDequantCodes + threadIdx.x * 8;
  T* dst = out + blockIdx.y * per_page + at;
  uint2 w[kTurns];
  float s[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t j = at + i * 8 * kDequantThreads;
    w[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (good) {
      w[i] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.pages) +
                                             page * per_page + j);
      s[i] = c.scales[page * c.kv_heads * 2 + j / (kBlock * c.head_dim)];
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    Vec8 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t pair = (e < 2 ? w[i].x : w[i].y) >> (16 * (e % 2));
      v.w[e] = pack<T>(make_float2((float(pair & 0xffu) - 128.f) * s[i],
                                   (float(pair >> 8 & 0xffu) - 128.f) * s[i]));
    }
    if (!good) v = Vec8{};
    store8(dst + i * 8 * kDequantThreads, v);
  }
}

template <typename T, int D>
void launch_t(const Args& a, unsigned flags, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  constexpr int kWarps = kThreads<D> / 32;
  cfg.gridDim = dim3(unsigned(a.block_items * a.c.kv_heads + (a.n_tokens * kParts + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads<D>);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, rope_append_kernel<T, D>, a);
}

}  // namespace

qlin_status launch_rope_table(float* table, int64_t n_positions, int rot_dim, double base,
                              double factor, double short_wavelength, double long_wavelength,
                              cudaStream_t st) {
  const int64_t n = n_positions * (rot_dim / 2);
  rope_table_kernel<<<unsigned((n + 255) / 256), 256, 0, st>>>(
      table, n_positions, rot_dim / 2, base, factor, short_wavelength, long_wavelength);
  return check_launch("qlin_rope_table");
}

qlin_status launch_rope_append(const void* qkv, int64_t qkv_stride, void* q_out,
                               const float* table, int64_t n_positions, int rot_dim,
                               int interleaved, const qlin_kv_cache& c, const int32_t* starts,
                               int64_t n_tokens, int q_heads, unsigned flags, cudaStream_t st) {
  // a slot with n new tokens completes at most (63 + n)/64 blocks, and at most n
  const int64_t most = n_tokens / kBlock + c.slots;
  const Args a = {qkv,    qkv_stride, q_out,   table,    n_positions,
                  rot_dim, interleaved, c,      starts,   n_tokens,
                  q_heads, n_tokens < most ? n_tokens : most};
  if (c.dtype == QLIN_F16)
    c.head_dim == 64 ? launch_t<__half, 64>(a, flags, st) : launch_t<__half, 128>(a, flags, st);
  else
    c.head_dim == 64 ? launch_t<__nv_bfloat16, 64>(a, flags, st)
                     : launch_t<__nv_bfloat16, 128>(a, flags, st);
  return check_launch("qlin_rope_append");
}

qlin_status launch_cache_dequant(const qlin_kv_cache& c, const int32_t* page_ids, int64_t n,
                                 void* out, cudaStream_t st) {
  const int64_t per_page = int64_t(c.kv_heads) * 2 * kBlock * c.head_dim;
  const int64_t elem = 2;
  for (int64_t at = 0; at < n; at += 32768) {  // the grid's second axis ends at 65535
    const dim3 grid(unsigned(per_page / kDequantCodes),
                    unsigned(n - at < 32768 ? n - at : 32768));
    void* dst = static_cast<uint8_t*>(out) + at * per_page * elem;
    if (c.dtype == QLIN_F16)
      cache_dequant_kernel<<<grid, kDequantThreads, 0, st>>>(c, page_ids + at,
                                                             static_cast<__half*>(dst));
    else
      cache_dequant_kernel<<<grid, kDequantThreads, 0, st>>>(c, page_ids + at,
                                                             static_cast<__nv_bfloat16*>(dst));
  }
  return check_launch("qlin_cache_dequant");
}

cudaError_t rope_take_device_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_rope_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace qlin
