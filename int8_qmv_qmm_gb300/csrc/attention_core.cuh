// What the attention kernels share: the arguments, the 16-bit products on 8-bit
// codes, and one warp's running softmax over blocks of the cache.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j),  j <= the row's position
//
// With k_j = s_k c_j and v_j = s_v c_j inside a block (c: whole numbers, -127 ..
// 127, exact in 16-bit floating point), the scales leave the products:
//   score = (scale * s_k) * (q . c_j)         out += s_v * sum_j p_j c_j
// so both products run on codes, with float32 sums, and only p is rounded.
#pragma once

#include <cmath>
#include <type_traits>

#include "kv_cache.cuh"

namespace qlin {
namespace attention {

constexpr int kRows = 16;       // rows (new token, query head) of a warp's tile
constexpr int kSplitRows = 64;  // slots with more rows go to the tile kernel

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

__device__ __forceinline__ uint32_t half2_bits(__half2 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t bf162_bits(__nv_bfloat162 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}

// Four codes (a word) as two pairs of 16-bit values c - 128, exactly.
// f16: 0x6400 | c is 1024 + c, minus 1152.  bf16 has 7 fraction bits, so the
// code's top bit goes to the subtrahend: (128 + c%128) - (c < 128 ? 256 : 128).
template <typename T>
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t& lo, uint32_t& hi);
template <>
__device__ __forceinline__ void widen_codes<__half>(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t bias = 0x64806480u;
  uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 k = *reinterpret_cast<const __half2*>(&bias);
  lo = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&a), k));
  hi = half2_bits(__hsub2(*reinterpret_cast<__half2*>(&b), k));
}
template <>
__device__ __forceinline__ void widen_codes<__nv_bfloat16>(uint32_t w, uint32_t& lo,
                                                           uint32_t& hi) {
  const uint32_t p[2] = {__byte_perm(w, 0u, 0x4140), __byte_perm(w, 0u, 0x4342)};
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t a = (p[i] & 0x007f007fu) | 0x43004300u, b = (~p[i] & 0x00800080u) | 0x43004300u;
    out[i] = bf162_bits(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                *reinterpret_cast<__nv_bfloat162*>(&b)));
  }
  lo = out[0];
  hi = out[1];
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

// The order of tokens and dimensions inside the products.  A product may sum
// its k axis in any order, and the columns of the scores may stand for any
// tokens, so both are chosen to make each thread's share of a block 16
// consecutive bytes.  Thread (g, t) = (lane/4, lane%4):
//   dimension of k step s, thread t:        64(s/4) + 16t + 4(s%4) + {0,1,2,3}
//   token of score tile j = 2s + h, column n: 16(n/2) + 4s + 2h + n%2
// and so a thread's scores of tiles 2s, 2s+1 are the tokens 16t + 4s + {0,1,2,3},
// which is k step s of the second product, whose operand it reads as 16
// consecutive tokens of a value row.
template <typename T, int D>
struct Warp {
  static constexpr int kQk = D / 16;  // k steps of the scores
  static constexpr int kPv = D / 8;   // column tiles of the output
  uint32_t q[kQk][4];
  float o[kPv][4];
  float m[2], l[2];  // of rows g and g + 8; scores in units of log2
  float unit;        // o counts in units of this: the largest value scale so far

  __device__ void init() {
#pragma unroll
    for (int i = 0; i < kPv; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    unit = 0.f;
  }

  // rows: [2] row pointers of this thread's two rows (null: zeros)
  __device__ void load_q(const T* r0, const T* r1, int t) {
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
      uint4 v[2][2] = {};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const T* src = r ? r1 : r0;
        if (src) {
          v[r][0] = *reinterpret_cast<const uint4*>(src + 64 * p + 16 * t);
          v[r][1] = *reinterpret_cast<const uint4*>(src + 64 * p + 16 * t + 8);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t w[8] = {v[r][0].x, v[r][0].y, v[r][0].z, v[r][0].w,
                               v[r][1].x, v[r][1].y, v[r][1].z, v[r][1].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          q[4 * p + s][r] = w[2 * s];
          q[4 * p + s][2 + r] = w[2 * s + 1];
        }
      }
    }
  }

  // Scores -> weighted probabilities (in place) with the running maximum; the
  // factors that the rows' sums so far take go to keep.  seen[r]: tokens of the
  // block that row r sees.  weight: what the probabilities are scaled by.
  template <int HALVES>
  __device__ void softmax(float (&s)[8][4], float scale, float weight, const int (&seen)[2],
                          bool mask, int t, float (&keep)[2]) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 2 * HALVES; ++e) s[j][e] *= scale;
    if (mask) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2 * HALVES; ++e)
          if (16 * t + 2 * j + (e & 1) >= seen[e >> 1]) s[j][e] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 2 * HALVES; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[j][e]);
    const float shift = log2f(weight), back = 1.f / weight;
#pragma unroll
    for (int r = 0; r < HALVES; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const float next = fmaxf(m[r], top[r]);
      const float base = next == -INFINITY ? 0.f : next;  // a row that sees nothing yet
      keep[r] = exp2_fast(m[r] - base);
      m[r] = next;
      const float from = base - shift;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = exp2_fast(s[j][2 * r + e] - from);
          s[j][2 * r + e] = p;
          sum += p;
        }
      l[r] = l[r] * keep[r] + sum * back;
    }
  }

  template <int HALVES>
  __device__ void rescale(const float (&keep)[2], float ratio) {
#pragma unroll
    for (int i = 0; i < kPv; ++i)
#pragma unroll
      for (int e = 0; e < 2 * HALVES; ++e) o[i][e] *= keep[e >> 1] * ratio;
  }

  // The factor from the old unit to the new, which is at least v.
  __device__ float raise_unit(float v) {
    const float next = fmaxf(unit, v);
    const float ratio = next > 0.f ? unit / next : 0.f;
    unit = next;
    return ratio;
  }

  // The scores of a complete block's 64 keys, in units of its key scale.
  __device__ void scores(const uint8_t* codes, float (&s)[8][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
      const uint8_t* row = codes + (16 * (g >> 1) + 2 * j + (g & 1)) * D + 16 * t;
#pragma unroll
      for (int p = 0; p < D / 64; ++p) {
        const uint4 w = *reinterpret_cast<const uint4*>(row + 64 * p);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          widen_codes<T>(words[i], b0, b1);
          mma<T>(s[j], q[4 * p + i], b0, b1);
        }
      }
    }
  }

  // Scores -> the second product's operand.  The probabilities enter it in f16
  // whatever T is: the codes are exact in f16, and it rounds p to 11 bits where
  // bf16 has 8.  HALVES = 1: rows 8 .. 15 of the tile are empty.
  template <int HALVES>
  __device__ void probabilities(float (&s)[8][4], uint32_t (&a)[4][4], float k_scale,
                                float v_scale, float scale, const int (&seen)[2], bool mask,
                                int t) {
    const float ratio = raise_unit(v_scale);
    // (a block whose values are all zero has scale 0: its codes are zero too; a
    // weight below f16's range makes every probability zero in it)
    const float weight = v_scale > 0.f ? fmaxf(v_scale / unit, 0x1p-60f) : 1.f;
    float keep[2] = {1.f, 1.f};
    softmax<HALVES>(s, scale * k_scale, weight, seen, mask, t, keep);
    rescale<HALVES>(keep, ratio);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          a[i][2 * h + r] = r < HALVES ? pack2<__half>(s[2 * i + h][2 * r], s[2 * i + h][2 * r + 1])
                                       : 0u;
  }

  // out += probabilities * the block's values (codes of D rows of 64 tokens)
  __device__ void values(const uint8_t* codes, const uint32_t (&a)[4][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < kPv; ++n) {
      const uint4 w = *reinterpret_cast<const uint4*>(codes + (8 * n + g) * kBlock + 16 * t);
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t b0, b1;
        widen_codes<__half>(words[i], b0, b1);
        mma<__half>(o[n], a[i], b0, b1);
      }
    }
  }

  // The tail: `count` tokens of T, the rest of its memory undefined.
  __device__ void tail(const T* kv, int count, float scale, const int (&seen)[2],
                                    int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
      const T* row = kv + (16 * (g >> 1) + 2 * j + (g & 1)) * D + 16 * t;
#pragma unroll
      for (int p = 0; p < D / 64; ++p) {
        const uint4 w0 = *reinterpret_cast<const uint4*>(row + 64 * p);
        const uint4 w1 = *reinterpret_cast<const uint4*>(row + 64 * p + 8);
        const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mma<T>(s[j], q[4 * p + i], words[2 * i], words[2 * i + 1]);
      }
    }
    const float ratio = raise_unit(1.f);
    float keep[2];
    softmax<2>(s, scale, 1.f, seen, true, t, keep);
    rescale<2>(keep, ratio);
    const float weight = 1.f / unit;
    // Undefined values must not meet the zeros of masked probabilities: 0 * NaN.
    uint32_t valid[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = 16 * t + 4 * i + 2 * h;
        valid[i][h] = tok + 1 < count ? 0xffffffffu : tok < count ? 0x0000ffffu : 0u;
      }
    // bf16 keeps only 8 bits of p, so what it leaves over goes through a second
    // product.
    constexpr bool kTwo = std::is_same<T, __nv_bfloat16>::value;
    uint32_t a[4][4], rest[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = s[2 * i + h][2 * r] * weight, p1 = s[2 * i + h][2 * r + 1] * weight;
          a[i][2 * h + r] = pack2<T>(p0, p1);
          if (kTwo)
            rest[i][2 * h + r] = pack2<T>(p0 - low_f32(a[i][2 * h + r]),
                                          p1 - high_f32(a[i][2 * h + r]));
        }
    kv += kBlock * D;
#pragma unroll
    for (int n = 0; n < kPv; ++n) {
      const T* row = kv + (8 * n + g) * kBlock + 16 * t;
      const uint4 w0 = *reinterpret_cast<const uint4*>(row);
      const uint4 w1 = *reinterpret_cast<const uint4*>(row + 8);
      const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b0 = words[2 * i] & valid[i][0], b1 = words[2 * i + 1] & valid[i][1];
        mma<T>(o[n], a[i], b0, b1);
        if (kTwo) mma<T>(o[n], rest[i], b0, b1);
      }
    }
  }
};

// Launchers of the two kernels (attention_split.cu, attention_tile.cu), and the
// status words that they set.
size_t split_workspace_size(int head_dim);
void launch_split(const Args& a, void* workspace, unsigned flags, cudaStream_t st);
void launch_tile(const Args& a, unsigned flags, cudaStream_t st);
cudaError_t split_take_status(unsigned* flags);
cudaError_t tile_take_status(unsigned* flags);

}  // namespace attention
}  // namespace qlin
