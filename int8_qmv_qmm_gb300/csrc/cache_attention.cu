// Attention of new tokens over the 8-bit key/value cache (qlin.h has the
// formats).
//
//   out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j),  j <= the row's position
//
// With k_j = s_k c_j and v_j = s_v c_j inside a block (c: whole numbers, -127 ..
// 127, exact in 16-bit floating point), the scales leave the products:
//   score = (scale * s_k) * (q . c_j)         out += s_v * sum_j p_j c_j
// so both products run on codes, with float32 sums, and only p is rounded.
//
// Simple form: one CTA for each 16 rows (a row is a new token and one of the
// query heads that share a key/value head) and key/value head.  Its warps take
// the blocks in turn, each with a running maximum and sum of its own
// (m16n8k16 products), and are joined at the end.

#include <cmath>
#include <type_traits>

#include "kv_cache.cuh"

namespace qlin {

__device__ unsigned int g_attention_status = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_attention_status, bit); }

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

  // Scores -> probabilities (in place) with the running maximum; returns the
  // factors that the two rows' sums so far take.  seen[r]: tokens of the block
  // that row r sees.
  __device__ void softmax(float (&s)[8][4], float scale, const int (&seen)[2], bool mask, int t,
                          float (&keep)[2]) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = s[j][e] * scale;
        if (mask && 16 * t + 2 * j + (e & 1) >= seen[e >> 1]) v = -INFINITY;
        s[j][e] = v;
        top[e >> 1] = fmaxf(top[e >> 1], v);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const float next = fmaxf(m[r], top[r]);
      const float base = next == -INFINITY ? 0.f : next;  // a row that sees nothing yet
      keep[r] = exp2f(m[r] - base);
      m[r] = next;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = exp2f(s[j][2 * r + e] - base);
          s[j][2 * r + e] = p;
          sum += p;
        }
      l[r] = l[r] * keep[r] + sum;
    }
  }

  __device__ void rescale(const float (&keep)[2], float ratio) {
    const float f[2] = {keep[0] * ratio, keep[1] * ratio};
#pragma unroll
    for (int i = 0; i < kPv; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] *= f[e >> 1];
  }

  // The factor from the old unit to the new, which is at least v.
  __device__ float raise_unit(float v) {
    const float next = fmaxf(unit, v);
    const float ratio = next > 0.f ? unit / next : 0.f;
    unit = next;
    return ratio;
  }

  // A complete block: codes of 64 keys and of D value rows.
  __device__ void block(const uint8_t* codes, float k_scale, float v_scale, float scale,
                        const int (&seen)[2], bool mask, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[8][4];
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
    float keep[2];
    softmax(s, scale * k_scale, seen, mask, t, keep);
    const float ratio = raise_unit(v_scale);
    rescale(keep, ratio);
    const float weight = unit > 0.f ? v_scale / unit : 0.f;
    // The probabilities enter in f16 whatever T is: the codes are exact in it,
    // and it rounds p to 11 bits where bf16 has 8.
    uint32_t a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          a[i][2 * h + r] =
              pack2<__half>(s[2 * i + h][2 * r] * weight, s[2 * i + h][2 * r + 1] * weight);
    codes += kBlock * D;
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
  __device__ void tail(const T* kv, int count, float scale, const int (&seen)[2], int lane) {
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
    float keep[2];
    softmax(s, scale, seen, true, t, keep);
    rescale(keep, raise_unit(1.f));
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

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const Args a) {
  __shared__ float s_o[kWarps][kRows][D + 4];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  grid_launch_dependents();
  grid_dependency_wait();
  const int kvh = blockIdx.y;
  int b = 0;
  int64_t tile = 0;
  if (!find_slot(a.c.slots, blockIdx.x, &b, &tile, [&](int s) -> int64_t {
        const SlotRows r = slot_rows(a.starts, a.c.lens, s, a.n_tokens);
        if (r.bad) report(kStatusRows);
        return (int64_t(r.n) * a.group + kRows - 1) / kRows;
      }))
    return;
  const SlotRows r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
  const int rows = r.n * a.group, r0 = int(tile) * kRows;
  const bool over = r.n > a.max_new;
  if (over && threadIdx.x == 0) report(kStatusMaxNew);
  Warp<T, D> w;
  w.init();
  const T* qp[2];
  int pos[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = r0 + g + 8 * i;
    qp[i] = row < rows ? static_cast<const T*>(a.q) + (r.row0 + row / a.group) * a.q_stride +
                             (kvh * a.group + row % a.group) * D
                       : nullptr;
    pos[i] = row < rows ? r.held + row / a.group : -1;
  }
  w.load_q(qp[0], qp[1], t);
  const int total = r.held + r.n, full = total / kBlock;
  const int last = r.held + (min(r0 + kRows, rows) - 1) / a.group;  // last position seen
  const int first = r.held + r0 / a.group;
  if (!over) {
    for (int j = warp; j <= last / kBlock; j += kWarps) {
      const int seen[2] = {pos[0] - j * kBlock + 1, pos[1] - j * kBlock + 1};
      if (j < full) {
        const int64_t page = page_of(a.c, b, j);
        if (page < 0) {
          if (lane == 0) report(kStatusPage);
          continue;
        }
        const int64_t at = page * a.c.kv_heads + kvh;
        w.block(static_cast<const uint8_t*>(a.c.pages) + at * 2 * kBlock * D, a.c.scales[2 * at],
                a.c.scales[2 * at + 1], a.scale_log2, seen, first < j * kBlock + kBlock - 1,
                lane);
      } else {
        w.tail(static_cast<const T*>(a.c.tail) +
                   (int64_t(b) * a.c.kv_heads + kvh) * 2 * kBlock * D,
               total - j * kBlock, a.scale_log2, seen, lane);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.l[i] += __shfl_xor_sync(0xffffffffu, w.l[i], 1);
    w.l[i] += __shfl_xor_sync(0xffffffffu, w.l[i], 2);
    if (t == 0) {
      s_m[warp][g + 8 * i] = w.m[i];
      s_l[warp][g + 8 * i] = w.l[i];
    }
  }
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_o[warp][g + 8 * (e >> 1)][8 * n + 2 * t + (e & 1)] = w.o[n][e] * w.unit;
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * D; i += blockDim.x) {
    const int row = i / D, d = i % D;
    if (r0 + row >= rows) break;
    float top = -INFINITY;
    for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_m[k][row]);
    float sum = 0.f, o = 0.f;
    for (int k = 0; k < kWarps; ++k) {
      const float f = s_m[k][row] == -INFINITY ? 0.f : exp2f(s_m[k][row] - top);
      sum += s_l[k][row] * f;
      o += s_o[k][row][d] * f;
    }
    static_cast<T*>(a.out)[((r.row0 + (r0 + row) / a.group) * a.q_heads + kvh * a.group +
                            (r0 + row) % a.group) *
                               D +
                           d] = Act<T>::from_f32_rn(sum > 0.f ? o / sum : 0.f);
  }
}

template <typename T, int D>
void launch_t(const Args& a, unsigned flags, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int64_t most = (a.n_tokens * a.group) / kRows + a.c.slots;  // tiles of all slots
  cfg.gridDim = dim3(unsigned(most), unsigned(a.c.kv_heads));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & QLIN_OVERLAP_PREVIOUS) ? 1 : 0;
  cudaLaunchKernelEx(&cfg, attention_kernel<T, D>, a);
}

}  // namespace

size_t cache_attention_workspace_size(int head_dim) {
  return head_dim == 64 || head_dim == 128 ? 256 : 0;
}

qlin_status launch_cache_attention(const void* q, int64_t q_stride, void* out,
                                   const qlin_kv_cache& c, const int32_t* starts,
                                   int64_t n_tokens, int q_heads, float scale, int max_new,
                                   void* workspace, unsigned flags, cudaStream_t st) {
  (void)workspace;
  const Args a = {q,
                  q_stride,
                  out,
                  c,
                  starts,
                  n_tokens,
                  q_heads,
                  q_heads / c.kv_heads,
                  scale * 1.4426950408889634f,
                  max_new};
  if (c.dtype == QLIN_F16)
    c.head_dim == 64 ? launch_t<__half, 64>(a, flags, st) : launch_t<__half, 128>(a, flags, st);
  else
    c.head_dim == 64 ? launch_t<__nv_bfloat16, 64>(a, flags, st)
                     : launch_t<__nv_bfloat16, 128>(a, flags, st);
  return check_launch("qlin_cache_attention");
}

cudaError_t attention_take_device_status(unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_attention_status, sizeof(v));
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(zero));
  *flags = v;
  return e;
}

}  // namespace qlin
