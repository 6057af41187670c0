// Rotary positions and the append to the 8-bit key/value cache (qlin.h has the
// formats), the table of cosines and sines, and the cache's reconstruction.
//
// One launch does two kinds of work:
//   token warps   one warp per new token: turns its queries and, where the
//                 token's block stays incomplete, its keys, which go with its
//                 values to the slot's tail;
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
// latency a decode step.  Angles come from a table made in 64 bits: at
// position 100000 a float32 angle would be off by up to 4e-3 radians.

#include <cmath>
#include <type_traits>

#include "kv_cache.cuh"

namespace qlin {

__device__ unsigned int g_rope_status = 0;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_rope_status, bit); }

template <typename T>
struct alignas(16) Vec8 {
  T v[8];
};

template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
  return *reinterpret_cast<const Vec8<T>*>(p);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& v) {
  *reinterpret_cast<Vec8<T>*>(p) = v;
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

// cs: the position's row of the table.
template <typename T>
__device__ __forceinline__ void rotate_unit(Vec8<T>& x, Vec8<T>& y, int u, int rot,
                                            bool interleaved, const float* cs) {
  if (16 * u >= rot) return;
  float t[16];
  const float4* p = reinterpret_cast<const float4*>(cs + 16 * u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = p[i];
    t[4 * i] = v.x, t[4 * i + 1] = v.y, t[4 * i + 2] = v.z, t[4 * i + 3] = v.w;
  }
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = Act<T>::to_f32(x.v[i]), b[i] = Act<T>::to_f32(y.v[i]);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn(a[2 * i], a[2 * i + 1], t[2 * i], t[2 * i + 1]);
      turn(b[2 * i], b[2 * i + 1], t[8 + 2 * i], t[8 + 2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(a[i], b[i], t[2 * i], t[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x.v[i] = Act<T>::from_f32_rn(a[i]), y.v[i] = Act<T>::from_f32_rn(b[i]);
}

// The code of v in a block of this scale.
__device__ __forceinline__ unsigned code_of(float v, float scale) {
  if (!(scale > 0.f)) return 128u;
  return unsigned(fminf(fmaxf(rintf(__fdiv_rn(v, scale)), -127.f), 127.f) + 128.f);
}

__device__ __forceinline__ float block_max(float v, float* partial) {
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = v;
  __syncthreads();
  v = partial[0];
  for (int i = 1; i < kWarps; ++i) v = fmaxf(v, partial[i]);
  return v;
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

// One new token's keys and values to the tail.
template <typename T, int D>
__device__ void token_to_tail(const Args& a, const T* row, int b, int pos, int unit0, int step) {
  const float* cs = a.table + int64_t(pos) * a.rot;
  const int at = pos % kBlock;
  for (int i = unit0; i < a.c.kv_heads * (D / 16); i += step) {
    const int h = i / (D / 16), u = i % (D / 16);
    T* tail = static_cast<T*>(a.c.tail) + (int64_t(b) * a.c.kv_heads + h) * 2 * kBlock * D;
    const T* k = row + (a.q_heads + h) * D;
    const T* v = row + (a.q_heads + a.c.kv_heads + h) * D;
    const Unit un = unit_of(u, a.rot, a.interleaved);
    Vec8<T> x = load8(k + un.at0), y = load8(k + un.at1);
    const Vec8<T> v0 = load8(v + 16 * u), v1 = load8(v + 16 * u + 8);
    rotate_unit(x, y, u, a.rot, a.interleaved, cs);
    store8(tail + at * D + un.at0, x);
    store8(tail + at * D + un.at1, y);
    T* vt = tail + kBlock * D;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      vt[(16 * u + e) * kBlock + at] = v0.v[e];
      vt[(16 * u + 8 + e) * kBlock + at] = v1.v[e];
    }
  }
}

template <typename T, int D>
__device__ void token_warp(const Args& a, int64_t t) {
  const int lane = threadIdx.x & 31;
  // the token's slot: the last one that starts at or before it
  int b = -1;
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
  const int pos = r.held + int(t - r.row0);
  const T* row = static_cast<const T*>(a.qkv) + t * a.qkv_stride;
  T* out = static_cast<T*>(a.q_out) + t * a.q_heads * D;
  const float* cs = a.table + int64_t(pos) * a.rot;
  for (int i = lane; i < a.q_heads * (D / 16); i += 32) {
    const int h = i / (D / 16), u = i % (D / 16);
    const Unit un = unit_of(u, a.rot, a.interleaved);
    Vec8<T> x = load8(row + h * D + un.at0), y = load8(row + h * D + un.at1);
    rotate_unit(x, y, u, a.rot, a.interleaved, cs);
    store8(out + h * D + un.at0, x);
    store8(out + h * D + un.at1, y);
  }
  const int total = r.held + r.n;
  const bool stays = pos / kBlock == total / kBlock;
  const bool left_to_block = total / kBlock > r.held / kBlock && r.held % kBlock;
  if (stays && !left_to_block) token_to_tail<T, D>(a, row, b, pos, lane, 32);
}

template <typename T, int D>
__device__ void block_cta(const Args& a, int64_t item, int h) {
  constexpr int kStride = kBlock + 2;  // of a staged value row: spreads the banks
  __shared__ T staged[D * kStride];
  __shared__ float partial[kWarps];
  __shared__ int s_slot, s_place;
  if (threadIdx.x < 32) {
    int b = -1;
    int64_t place = 0;
    const bool any = find_slot(a.c.slots, item, &b, &place, [&](int s) -> int64_t {
      const SlotRows r = slot_rows(a.starts, a.c.lens, s, a.n_tokens);
      return slot_fits(a, r) ? (int64_t(r.held) + r.n) / kBlock - r.held / kBlock : 0;
    });
    if (threadIdx.x == 0) s_slot = any ? b : -1, s_place = int(place);
  }
  __syncthreads();
  const int b = s_slot;
  if (b < 0) return;
  const SlotRows r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
  const int j = r.held / kBlock + s_place;
  const int old = j == r.held / kBlock ? r.held % kBlock : 0;  // tokens that the tail holds
  const int64_t page = page_of(a.c, b, j);
  if (page < 0 && threadIdx.x == 0) report(kStatusPage);
  T* tail = static_cast<T*>(a.c.tail) + (int64_t(b) * a.c.kv_heads + h) * 2 * kBlock * D;
  // rows of the block's new tokens: token i of the block is row first + i
  const int64_t first = r.row0 + int64_t(j) * kBlock - r.held;
  const T* qkv = static_cast<const T*>(a.qkv);

  // keys: each thread holds kUnits units of 16 elements
  constexpr int kUnits = kBlock * (D / 16) / kThreads;
  static_assert(kUnits * kThreads == kBlock * (D / 16), "units divide evenly");
  Vec8<T> kx[kUnits], ky[kUnits];
  float top = 0.f;
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int i = n * kThreads + threadIdx.x, tok = i / (D / 16), u = i % (D / 16);
    const Unit un = unit_of(u, a.rot, a.interleaved);
    if (tok < old) {
      kx[n] = load8(tail + tok * D + un.at0);
      ky[n] = load8(tail + tok * D + un.at1);
    } else {
      const T* k = qkv + (first + tok) * a.qkv_stride + (a.q_heads + h) * D;
      kx[n] = load8(k + un.at0);
      ky[n] = load8(k + un.at1);
      rotate_unit(kx[n], ky[n], u, a.rot, a.interleaved,
                  a.table + (int64_t(j) * kBlock + tok) * a.rot);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      top = fmaxf(top, fmaxf(fabsf(Act<T>::to_f32(kx[n].v[e])), fabsf(Act<T>::to_f32(ky[n].v[e]))));
    // values, transposed on the way
    T v[16];
    if (tok < old) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = tail[kBlock * D + (16 * u + e) * kBlock + tok];
    } else {
      const T* p = qkv + (first + tok) * a.qkv_stride + (a.q_heads + a.c.kv_heads + h) * D + 16 * u;
      const Vec8<T> v0 = load8(p), v1 = load8(p + 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v0.v[e], v[8 + e] = v1.v[e];
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) staged[(16 * u + e) * kStride + tok] = v[e];
  }
  const float k_scale = __fdiv_rn(block_max(top, partial), 127.f);  // (orders `staged` too)

  T vv[kUnits][16];
  top = 0.f;
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int i = n * kThreads + threadIdx.x, d = i / 4, t0 = (i % 4) * 16;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      vv[n][e] = staged[d * kStride + t0 + e];
      top = fmaxf(top, fabsf(Act<T>::to_f32(vv[n][e])));
    }
  }
  const float v_scale = __fdiv_rn(block_max(top, partial), 127.f);
  if (page >= 0) {
    uint8_t* codes = static_cast<uint8_t*>(a.c.pages) + (page * a.c.kv_heads + h) * 2 * kBlock * D;
    if (threadIdx.x == 0) {
      float* s = a.c.scales + (page * a.c.kv_heads + h) * 2;
      s[0] = k_scale;
      s[1] = v_scale;
    }
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int i = n * kThreads + threadIdx.x, tok = i / (D / 16), u = i % (D / 16);
      const Unit un = unit_of(u, a.rot, a.interleaved);
      uint32_t w[4] = {0, 0, 0, 0}, z[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e / 4] |= code_of(Act<T>::to_f32(kx[n].v[e]), k_scale) << (8 * (e % 4));
        w[2 + e / 4] |= code_of(Act<T>::to_f32(ky[n].v[e]), k_scale) << (8 * (e % 4));
      }
      *reinterpret_cast<uint2*>(codes + tok * D + un.at0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(codes + tok * D + un.at1) = make_uint2(w[2], w[3]);
      const int d = i / 4, t0 = (i % 4) * 16;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        z[e / 4] |= code_of(Act<T>::to_f32(vv[n][e]), v_scale) << (8 * (e % 4));
      *reinterpret_cast<uint4*>(codes + kBlock * D + d * kBlock + t0) =
          make_uint4(z[0], z[1], z[2], z[3]);
    }
  }
  // the new tail, where the old one had tokens of this block (all read above:
  // the barriers of block_max lie in between)
  const int total = r.held + r.n;
  if (old) {
    for (int tok = threadIdx.x / (D / 16); tok < total % kBlock; tok += kThreads / (D / 16)) {
      const int u = threadIdx.x % (D / 16), pos = total / kBlock * kBlock + tok;
      const T* row = qkv + (r.row0 + pos - r.held) * a.qkv_stride;
      const Unit un = unit_of(u, a.rot, a.interleaved);
      const T* k = row + (a.q_heads + h) * D;
      const T* v = row + (a.q_heads + a.c.kv_heads + h) * D + 16 * u;
      Vec8<T> x = load8(k + un.at0), y = load8(k + un.at1);
      const Vec8<T> v0 = load8(v), v1 = load8(v + 8);
      rotate_unit(x, y, u, a.rot, a.interleaved, a.table + int64_t(pos) * a.rot);
      store8(tail + tok * D + un.at0, x);
      store8(tail + tok * D + un.at1, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        tail[kBlock * D + (16 * u + e) * kBlock + tok] = v0.v[e];
        tail[kBlock * D + (16 * u + 8 + e) * kBlock + tok] = v1.v[e];
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const Args a) {
  grid_launch_dependents();
  grid_dependency_wait();
  // block CTAs first: they take longer
  const int64_t blocks = a.block_items * a.c.kv_heads;
  if (blockIdx.x < blocks) {
    block_cta<T, D>(a, blockIdx.x / a.c.kv_heads, blockIdx.x % a.c.kv_heads);
  } else {
    const int64_t t = (blockIdx.x - blocks) * kWarps + (threadIdx.x >> 5);
    if (t < a.n_tokens) token_warp<T, D>(a, t);
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
template <typename T>
__global__ void __launch_bounds__(256)
    cache_dequant_kernel(const qlin_kv_cache c, const int32_t* __restrict__ ids, T* out) {
  const int64_t per_page = int64_t(c.kv_heads) * 2 * kBlock * c.head_dim;
  const int64_t page = ids[blockIdx.y];
  const bool good = page >= 0 && page < c.n_pages;
  if (!good && blockIdx.x == 0 && threadIdx.x == 0) report(kStatusPage);
  const int64_t i = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * 16;
  if (i >= per_page) return;
  T* dst = out + blockIdx.y * per_page + i;
  Vec8<T> v[2];
  if (good) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.pages) +
                                                    page * per_page + i);
    const float s = c.scales[page * c.kv_heads * 2 + i / (kBlock * c.head_dim)];
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 16; ++e)
      v[e / 8].v[e % 8] = Act<T>::from_f32_rn(
          (float((words[e / 4] >> (8 * (e % 4))) & 0xffu) - 128.f) * s);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e / 8].v[e % 8] = Act<T>::from_f32_rn(0.f);
  }
  store8(dst, v[0]);
  store8(dst + 8, v[1]);
}

template <typename T, int D>
void launch_t(const Args& a, unsigned flags, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.block_items * a.c.kv_heads + (a.n_tokens + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
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
    const dim3 grid(unsigned((per_page / 16 + 255) / 256),
                    unsigned(n - at < 32768 ? n - at : 32768));
    void* dst = static_cast<uint8_t*>(out) + at * per_page * elem;
    if (c.dtype == QLIN_F16)
      cache_dequant_kernel<<<grid, 256, 0, st>>>(c, page_ids + at, static_cast<__half*>(dst));
    else
      cache_dequant_kernel<<<grid, 256, 0, st>>>(c, page_ids + at,
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
