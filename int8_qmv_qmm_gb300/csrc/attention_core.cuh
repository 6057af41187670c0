// What the attention kernels share: the arguments, the 16-bit products on 8-bit
// codes, and one warp's running softmax over blocks of the cache.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j),  j <= the row's position
//
// With k_j = s_k c_j and v_j = s_v c_j inside a block (c: whole numbers, -127 ..
// 127, exact in 16-bit floating point), the scales leave the products:
//   score = (scale * s_k) * (q . c_j)         out += sum_j (s_v p_j) c_j
// so both products run on codes, with float32 sums, and only s_v p is rounded (to
// f16).  s_v goes into the exponent and into the running maximum,
//   s_v p_j = exp2(score + log2 s_v - m),  m the largest score + log2 s_v so far
// so that a rounding is 2^-11 of a token's own weight, or 2^-25 of the largest so
// far, whatever the blocks' scales are: a block of large values that gets no
// probability takes nothing from the others.  (With the values' scales relative to
// the largest of them, blocks 2^26 apart lost the smaller one.)  The denominator
// takes the weights back.
#pragma once

#include <cmath>
#include <type_traits>

#include "kv_cache.cuh"

namespace qlin {
namespace attention {

// Slots with more rows go to the tile kernel.  The split kernel's time grows with the
// rows, 8 of them a pass over the cache, the tile kernel's does not up to 256, but it
// starts behind: by 13 to 20 us with f16, 40 to 70 with a bf16 tail, which its widening
// warps go over twice.  Split against tile, us, 8 key/value heads, caches flushed:
//     slots x tokens        32 rows     64 rows     96 rows    128 rows
//     1 x 400,  f16 64     15 / 28     15 / 28     17 / 29     19 / 28
//               f16 128    17 / 39     19 / 39     19 / 38     20 / 39
//               bf16 64    17 / 55     17 / 54     19 / 55     19 / 55
//               bf16 128   17 / 90     19 / 92     21 / 90     21 / 90
//     8 x 8000, f16 64     66 / 92    113 / 92    160 / 92    207 / 92
//               f16 128   100 / 114   151 / 114   213 / 116   277 / 114
//               bf16 64    67 / 120   115 / 120   163 / 120   210 / 120
//               bf16 128  101 / 169   153 / 170   218 / 170   283 / 172
//     32 x 8000, f16 64   216 / 247   394 / 247   572 / 247   765 / 250
//               f16 128   370 / 314   568 / 315   791 / 317  1234 / 317
//               bf16 64   218 / 299   399 / 299   584 / 299   773 / 300
//               bf16 128  369 / 420   573 / 424   799 / 425  1221 / 425
// The rule goes by rows alone, since the lengths are on the device only: 64 serves short
// caches and bf16; many long f16 caches would want 32.
constexpr int kSplitRows = 64;

struct Args {
  const void* q;
  int64_t q_stride;
  void* out;
  qlin_kv_cache c;
  const int32_t* starts;
  int64_t n_tokens;
  int q_heads, group;
  float scale_log2;
  int max_new;
};

// D += A * B, A 16x16 (row), B 16x8 (col), f32 accumulators.
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                   uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp, exact at 0 and -infinity
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a row's sums are multiplied by at the end: 1 over its denominator; 0 for a row
// that saw nothing.  A NaN stays one, however the work was cut.
__device__ __forceinline__ float share_of(float l) { return l == 0.f ? 0.f : 1.f / l; }

__device__ __forceinline__ uint32_t half2_bits(__half2 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t bf162_bits(__nv_bfloat162 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}

// Four codes (a word) as two pairs of f16 values c - 128, exactly: 0x6400 | c is
// 1024 + c, minus 1152.
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t bias = 0x64806480u;
  uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 k = *reinterpret_cast<const __half2*>(&bias);
  lo = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&a), k));
  hi = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&b), k));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  return half2_bits(__floats2half2_rn(a, b));
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  return bf162_bits(__floats2bfloat162_rn(a, b));
}
__device__ __forceinline__ float low_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Transposes an 8x8 matrix of 16-bit values held as rows lane/4, columns
// 2(lane%4) + {0, 1}.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// The logarithm of a block's value scale, for the exponents; the denominator takes it
// back by exp2(-it).  A block whose values are all zero has scale 0, and any weight will
// do: its codes are zero too.  Scales below 2^-100 weigh as that (the sums of values
// below 2^-93 are off by as much).  Infinity, of a block that is not finite, makes the
// rows that see it NaN: infinite scores less an infinite maximum.
__device__ __forceinline__ float weight_log2(float v_scale) {
  const float w = v_scale > 0.f ? fmaxf(v_scale, 0x1p-100f) : 0x1p-60f;
  return log2_fast(v_scale == v_scale ? w : INFINITY);
}

// One warp's attention of 8 rows over blocks of the cache.
//
// Tokens (scores) and dimensions (outputs) are the 16 rows of the products and
// the query rows their 8 columns, so that a decode step's few rows fill the
// products, and a block's codes are widened once for all of them:
//   S^T [64 x 8]  = keys [64 x D] . q^T [D x 8]
//   O^T [D x 8]  += values^T [D x 64] . P^T [64 x 8]
// A product may sum its k axis in any order, and the rows of S^T may stand for
// any tokens; both are chosen to make each thread's share of a key or value
// row 16 consecutive bytes.  Thread (g, t) = (lane/4, lane%4):
//   dimension of k step s, thread t:   64(s/4) + 16t + 4(s%4) + {0,1,2,3}
//   token of score tile i, its row r:  16((r%8)/2) + 4i + 2(r/8) + r%2
// so that k step i of the second product, thread t, is the tokens
// 16t + 4i + {0,1,2,3} of a value row; S^T's fragments become P^T's by 8x8
// transposes in registers.
//
// Both products take f16 whatever T is: codes are exact in it, and it rounds p
// to 11 bits where bf16 has 8.  bf16 queries are scaled by a power of two for
// each row, to a largest magnitude of 2^14 .. 2^15: exact down to 2^-28 of it.
template <typename T, int D>
struct Warp {
  static constexpr int kQk = D / 16;  // k steps of the scores, row tiles of the output
  uint32_t q[kQk][2];
  float o[kQk][4];
  float factor[2];  // scores to units of log2, without the key scale
  float m[2], l[2];  // of rows 2t + {0, 1}; l over this lane's tokens

  __device__ void init() {
#pragma unroll
    for (int i = 0; i < kQk; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // A query row's fragments, in T.
  __device__ static void load_row(const T* src, uint32_t (&w)[D / 8], int t) {
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
      uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
      if (src) {
        v0 = *reinterpret_cast<const uint4*>(src + 64 * p + 16 * t);
        v1 = *reinterpret_cast<const uint4*>(src + 64 * p + 16 * t + 8);
      }
      w[8 * p + 0] = v0.x, w[8 * p + 1] = v0.y, w[8 * p + 2] = v0.z, w[8 * p + 3] = v0.w;
      w[8 * p + 4] = v1.x, w[8 * p + 5] = v1.y, w[8 * p + 6] = v1.z, w[8 * p + 7] = v1.w;
    }
  }

  // row: row g of the tile (null: zeros).  The fragments are T until
  // prepare_q.
  __device__ void load_q(const T* row, int lane) {
    uint32_t w[D / 8];
    load_row(row, w, lane & 3);
#pragma unroll
    for (int s = 0; s < kQk; ++s) {
      q[s][0] = w[2 * s];
      q[s][1] = w[2 * s + 1];
    }
  }

  __device__ void prepare_q(float scale, int lane) {
    const int t = lane & 3;
    float back = scale;
    if (std::is_same<T, __nv_bfloat16>::value) {
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < kQk; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          top = fmaxf(top, fmaxf(fabsf(low_f32(q[s][h])), fabsf(high_f32(q[s][h]))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = int(__float_as_uint(top) >> 23) - 127 - 14;  // q * 2^-e is below 2^15
      e = max(-100, min(113, e));
      const float down = __uint_as_float(uint32_t(127 - e) << 23);
      back = scale * __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
      for (int s = 0; s < kQk; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q[s][h] = pack2<__half>(low_f32(q[s][h]) * down, high_f32(q[s][h]) * down);
    }
    // row g's factor, to the lanes that hold the row's scores
    factor[0] = __shfl_sync(0xffffffffu, back, 8 * t);
    factor[1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
  }

  // Scores (times scale and the rows' factors) -> weighted probabilities, in
  // place, with the running maximum; the factors that the rows' sums so far take
  // go to keep.  shift: the logarithm of the block's weight.  seen[r]: tokens of the
  // block that row 2t + r sees.
  __device__ void softmax(float (&s)[4][4], const float (&scale)[2], float shift,
                          const int (&seen)[2], bool mask, int g, float (&keep)[2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = fmaf(s[i][e], scale[e & 1], shift);
    if (mask) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * (g >> 1) + 4 * i + 2 * (e >> 1) + (g & 1) >= seen[e & 1])
            s[i][e] = -INFINITY;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = fmaxf(s[0][r], s[0][2 + r]);
#pragma unroll
      for (int i = 1; i < 4; ++i) top = fmaxf(top, fmaxf(s[i][r], s[i][2 + r]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float next = fmaxf(m[r], top);
      const float base = next == -INFINITY ? 0.f : next;  // a row that sees nothing yet
      keep[r] = exp2_fast(m[r] - base);
      m[r] = next;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p = exp2_fast(s[i][2 * h + r] - base);
          s[i][2 * h + r] = p;
          sum += p;
        }
      l[r] = l[r] * keep[r] + sum * exp2_fast(-shift);
    }
  }

  __device__ void rescale(const float (&keep)[2]) {
#pragma unroll
    for (int i = 0; i < kQk; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] *= keep[e & 1];
  }

  // The scores of a complete block's 64 keys, in units of its key scale.
  __device__ void scores(const uint8_t* codes, float (&s)[4][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
      const uint8_t* row = codes + (16 * (g >> 1) + 4 * i + (g & 1)) * D + 16 * t;
#pragma unroll
      for (int p = 0; p < D / 64; ++p) {
        const uint4 w0 = *reinterpret_cast<const uint4*>(row + 64 * p);
        const uint4 w1 = *reinterpret_cast<const uint4*>(row + 2 * D + 64 * p);
        const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t a[4];
          widen_codes(x0[k], a[0], a[2]);
          widen_codes(x1[k], a[1], a[3]);
          mma<__half>(s[i], a, q[4 * p + k][0], q[4 * p + k][1]);
        }
      }
    }
  }

  // Scores -> the second product's operand.
  __device__ void probabilities(float (&s)[4][4], uint32_t (&b)[4][2], float k_scale,
                                float v_scale, const int (&seen)[2], bool mask, int lane) {
    float keep[2], scale[2];
    scale[0] = factor[0] * k_scale, scale[1] = factor[1] * k_scale;
    softmax(s, scale, weight_log2(v_scale), seen, mask, lane >> 2, keep);
    rescale(keep);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        b[i][h] = transpose8(pack2<__half>(s[i][2 * h], s[i][2 * h + 1]));
  }

  // out += probabilities * the block's values (codes of D rows of 64 tokens)
  __device__ void values(const uint8_t* codes, const uint32_t (&b)[4][2], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < kQk; ++i) {
      const uint8_t* row = codes + (16 * i + g) * kBlock + 16 * t;
      const uint4 w0 = *reinterpret_cast<const uint4*>(row);
      const uint4 w1 = *reinterpret_cast<const uint4*>(row + 8 * kBlock);
      const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[4];
        widen_codes(x0[k], a[0], a[2]);
        widen_codes(x1[k], a[1], a[3]);
        mma<__half>(o[i], a, b[k][0], b[k][1]);
      }
    }
  }

  // The first of the tail's tokens from about `from` on with a value that is not
  // finite, else count.
  __device__ static int first_lost(const T* values, int from, int count, int lane) {
    constexpr uint32_t kExponent = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    constexpr uint32_t kOne = kExponent & -kExponent;  // carries out of a full exponent
    const unsigned g0 = unsigned(from) / 8, groups = unsigned(count - 1) / 8 - g0 + 1;
    int lost = count;
#pragma unroll 4
    for (unsigned u = lane; u < D * groups; u += 32) {  // 8 tokens of a dimension each
      const unsigned t0 = 8 * (g0 + u % groups);
      const T* at = values + u / groups * kBlock + t0;
      const uint4 v = *reinterpret_cast<const uint4*>(at);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t any = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= (w[e] & kExponent * 0x10001u) + kOne * 0x10001u;
      if (any & 0x80008000u) {
#pragma unroll 1
        for (int e = 0; e < 8; ++e)
          if ((reinterpret_cast<const uint16_t*>(at)[e] & kExponent) == kExponent)
            lost = min(lost, int(t0) + e);
      }
    }
    return __reduce_min_sync(0xffffffffu, lost);
  }

  // The tail: `count` tokens of T, the rest of its memory undefined.  Products
  // in T (the queries come from memory again: q is f16).  All rows see its first
  // `common` tokens.  A value of the others that is not finite must not reach, as 0
  // times it, the rows that do not see it: values from its token on are left out, and
  // the rows that see it are NaN.  (Looking for one in the whole tail took 31.0 us for
  // 12 x 3 drafts, beside each product 33.0; 30.1 without.)
  __device__ void tail(const T* kv, int count, const T* q_row, float scale_log2,
                       const int (&seen)[2], int common, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[4][4];
    uint32_t w[D / 8];
    load_row(q_row, w, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
      const T* row = kv + (16 * (g >> 1) + 4 * i + (g & 1)) * D + 16 * t;
#pragma unroll
      for (int p = 0; p < D / 64; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // two k steps to a load
          const uint4 v0 = *reinterpret_cast<const uint4*>(row + 64 * p + 8 * h);
          const uint4 v1 = *reinterpret_cast<const uint4*>(row + 2 * D + 64 * p + 8 * h);
          const uint32_t a0[4] = {v0.x, v1.x, v0.y, v1.y}, a1[4] = {v0.z, v1.z, v0.w, v1.w};
          mma<T>(s[i], a0, w[8 * p + 4 * h], w[8 * p + 4 * h + 1]);
          mma<T>(s[i], a1, w[8 * p + 4 * h + 2], w[8 * p + 4 * h + 3]);
        }
    }
    float keep[2], scale[2];
    scale[0] = scale[1] = scale_log2;
    softmax(s, scale, 0.f, seen, true, g, keep);
    rescale(keep);
    const int lost =
        common < count ? first_lost(kv + kBlock * D, max(common, 0), count, lane) : count;
    if (lost < count) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (seen[r] > lost) l[r] = NAN;
    }
    // bf16 keeps only 8 bits of p, so what it leaves over goes through a second
    // product.
    constexpr bool kTwo = std::is_same<T, __nv_bfloat16>::value;
    uint32_t b[4][2], rest[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = s[i][2 * h], p1 = s[i][2 * h + 1];
        const uint32_t v = pack2<T>(p0, p1);
        b[i][h] = transpose8(v);
        if (kTwo) rest[i][h] = transpose8(pack2<T>(p0 - low_f32(v), p1 - high_f32(v)));
      }
    // Undefined values must not meet the zeros of masked probabilities: 0 * NaN.
    uint32_t valid[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = 16 * t + 4 * k + 2 * h;
        valid[k][h] = tok + 1 < lost ? 0xffffffffu : tok < lost ? 0x0000ffffu : 0u;
      }
    kv += kBlock * D;
#pragma unroll
    for (int i = 0; i < kQk; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const T* row = kv + (16 * i + g) * kBlock + 16 * t + 8 * h;
        const uint4 v0 = *reinterpret_cast<const uint4*>(row);
        const uint4 v1 = *reinterpret_cast<const uint4*>(row + 8 * kBlock);
        const uint32_t a[2][4] = {{v0.x, v1.x, v0.y, v1.y}, {v0.z, v1.z, v0.w, v1.w}};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int k = 2 * h + c;
          const uint32_t av[4] = {a[c][0] & valid[k][0], a[c][1] & valid[k][0],
                                  a[c][2] & valid[k][1], a[c][3] & valid[k][1]};
          mma<T>(o[i], av, b[k][0], b[k][1]);
          if (kTwo) mma<T>(o[i], av, rest[k][0], rest[k][1]);
        }
      }
  }
};

// Launchers of the two kernels (attention_split.cu, attention_tile.cu), and the
// status words that they set.  The split kernel's parts are joined by its own launch
// (`join`) or by the tile kernel's, with its pieces.
size_t split_workspace_size(int head_dim);
cudaError_t launch_split(const Args& a, void* workspace, bool join, unsigned flags,
                         cudaStream_t st);
size_t tile_workspace_size(int head_dim);
cudaError_t launch_tile(const Args& a, void* workspace, void* split_workspace, cudaStream_t st);
cudaError_t split_take_status(unsigned* flags);
cudaError_t tile_take_status(unsigned* flags);

}  // namespace attention
}  // namespace qlin
