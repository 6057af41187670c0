// What the tensor-core products on packed weights share: the reconstruction of a
// weight tile's rows into tensor memory as the MMA's A operand, and tensor maps.
#pragma once

#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "device_common.cuh"
#include "qlin_internal.h"
#include "sm100_ptx.cuh"

namespace qlin {
namespace {

constexpr int kBM = 128;          // weight rows per tile (MMA M)
constexpr int kBK = 64;           // k per stage (one group)

// D (TMEM, f32) += A (TMEM: row i in lane i, K along columns, two 16-bit
// elements per 32-bit column, element k in the low half) * B (shared memory
// descriptor); M = 128, accumulate = 0 overwrites D.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Each thread of the warp writes 32 consecutive 32-bit columns of its own TMEM
// lane (lane = the warp's lane quarter * 32 + lane id, taken from taddr).
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Wait until this thread's tcgen05.st have completed.
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int BITS>
struct Geo {
  static constexpr int kWordsPerGroup = kBK * BITS / 32;           // 8 or 16
  static constexpr int kPackedRowBytes = kWordsPerGroup * 4;       // 32 or 64
  static constexpr int kPackedBytes = kBM * kPackedRowBytes;       // 4 or 8 KB
};

// Operands per weight in the A slot: 1 (float16: w_hat), 2 (bfloat16: hi and
// the residual lo, see lo_pair).
template <typename AT>
struct OperandSplit {
  static constexpr int value = std::is_same<AT, __nv_bfloat16>::value ? 2 : 1;
};

// ---- unpack + dequantise one 16-bit pair: returns (w_hat[2j], w_hat[2j+1])
template <typename AT>
__device__ __forceinline__ uint32_t fma_pair(uint32_t magic_pair, uint32_t s2, uint32_t b2) {
  using T2 = typename Act<AT>::T2;
  const uint32_t mq = Act<AT>::kMagic2;
  T2 v = *reinterpret_cast<const T2*>(&magic_pair);
  const T2 m = *reinterpret_cast<const T2*>(&mq);
  const T2 q = __hsub2(v, m);  // exact: both are small integers plus the magic
  const T2 r = __hfma2(q, *reinterpret_cast<const T2*>(&s2), *reinterpret_cast<const T2*>(&b2));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 8 consecutive codes of a 4-bit word -> 8 reconstructed 16-bit weights.
template <typename AT>
__device__ __forceinline__ uint4 dequant_word4(uint32_t w, uint32_t s2, uint32_t b2) {
  const uint32_t sh = w >> 4;
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // low half <- byte j of w (code 2j in bits 0..3), high half <- byte j of
    // w >> 4 (code 2j+1 in bits 16..19)
    const uint32_t sel = uint32_t(j) | (uint32_t(j) << 4) | (uint32_t(4 + j) << 8) |
                         (uint32_t(4 + j) << 12);
    const uint32_t t = __byte_perm(w, sh, sel);
    out[j] = fma_pair<AT>((t & 0x000F000Fu) | Act<AT>::kMagic2, s2, b2);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// 4 codes of an 8-bit word -> 2 pairs.
template <typename AT>
__device__ __forceinline__ void dequant_word8(uint32_t w, uint32_t s2, uint32_t b2,
                                              uint32_t& p0, uint32_t& p1);

template <>
__device__ __forceinline__ void dequant_word8<__half>(uint32_t w, uint32_t s2, uint32_t b2,
                                                      uint32_t& p0, uint32_t& p1) {
  // 0x64 in the high byte of each half: 1024 + code, exact for codes < 1024
  p0 = fma_pair<__half>(__byte_perm(w, 0x64646464u, 0x4140u), s2, b2);
  p1 = fma_pair<__half>(__byte_perm(w, 0x64646464u, 0x4342u), s2, b2);
}

template <>
__device__ __forceinline__ void dequant_word8<__nv_bfloat16>(uint32_t w, uint32_t s2, uint32_t b2,
                                                             uint32_t& p0, uint32_t& p1) {
  // bfloat16 has 8 significant bits, too few for 128 + code; go through f32:
  // 2^23 + code is exact, the subtraction is exact, and the code (< 256) is
  // exact in bfloat16.
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | uint32_t(i))) - 8388608.0f;
  const __nv_bfloat162 q01 = __floats2bfloat162_rn(f[0], f[1]);
  const __nv_bfloat162 q23 = __floats2bfloat162_rn(f[2], f[3]);
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2);
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&b2);
  const __nv_bfloat162 r0 = __hfma2(q01, s, b), r1 = __hfma2(q23, s, b);
  p0 = *reinterpret_cast<const uint32_t*>(&r0);
  p1 = *reinterpret_cast<const uint32_t*>(&r1);
}

// ---- bfloat16 residual operand
// For a pair of weights with codes q (exact, as float), scale s and bias b in
// float32, and hi = RNE_bf16(q*s + b) (the pair as computed above):
//   d  = RNE_f32(q*s + b) - hi          (exact: the two are within 2^-8)
//   lo = RZ_bf16(RNE_f32(d * (1 - 2^-9)))
// Then |hi + lo - (q*s + b)| <= about 2^-15 |q*s + b|, and |lo| stays below
// half a bfloat16 step of hi (the factor keeps it there when the float32
// rounding lands exactly on a midpoint), so hi + lo, accumulated in float32
// and rounded to bfloat16, is hi again: a one-hot x still reproduces the
// reconstruction bit for bit.
__device__ __forceinline__ uint32_t lo_pair(float2 q, float2 s, float2 b, uint32_t hi) {
  const float2 fw = __ffma2_rn(q, s, b);
  const float2 h = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
  const float2 d = __ffma2_rn(h, make_float2(-1.0f, -1.0f), fw);
  const float2 dc = __fmul2_rn(d, make_float2(0.998046875f, 0.998046875f));
  uint32_t r;
  // the first source goes to the upper half
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(dc.y), "f"(dc.x));
  return r;
}

// 8 codes of a 4-bit word -> hi and lo of 8 bfloat16 weights.
__device__ __forceinline__ void dequant_word4_split(uint32_t w, uint32_t s2, uint32_t b2, float2 sf,
                                                    float2 bf, uint32_t (&hi)[4],
                                                    uint32_t (&lo)[4]) {
  const uint32_t sh = w >> 4;
  const uint32_t mq = Act<__nv_bfloat16>::kMagic2;
  const __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&mq);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t sel = uint32_t(j) | (uint32_t(j) << 4) | (uint32_t(4 + j) << 8) |
                         (uint32_t(4 + j) << 12);
    const uint32_t mp = (__byte_perm(w, sh, sel) & 0x000F000Fu) | Act<__nv_bfloat16>::kMagic2;
    const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&mp), m);
    const __nv_bfloat162 r = __hfma2(q, *reinterpret_cast<const __nv_bfloat162*>(&s2),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b2));
    const uint32_t qb = *reinterpret_cast<const uint32_t*>(&q);
    hi[j] = *reinterpret_cast<const uint32_t*>(&r);
    lo[j] = lo_pair(make_float2(__uint_as_float(qb << 16), __uint_as_float(qb & 0xffff0000u)), sf,
                    bf, hi[j]);
  }
}

// 4 codes of an 8-bit word -> hi and lo of 4 bfloat16 weights (two pairs).
__device__ __forceinline__ void dequant_word8_split(uint32_t w, uint32_t s2, uint32_t b2, float2 sf,
                                                    float2 bf, uint32_t& h0, uint32_t& h1,
                                                    uint32_t& l0, uint32_t& l1) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | uint32_t(i))) - 8388608.0f;
  const __nv_bfloat162 q01 = __floats2bfloat162_rn(f[0], f[1]);
  const __nv_bfloat162 q23 = __floats2bfloat162_rn(f[2], f[3]);
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2);
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&b2);
  const __nv_bfloat162 r0 = __hfma2(q01, s, b), r1 = __hfma2(q23, s, b);
  h0 = *reinterpret_cast<const uint32_t*>(&r0);
  h1 = *reinterpret_cast<const uint32_t*>(&r1);
  l0 = lo_pair(make_float2(f[0], f[1]), sf, bf, h0);
  l1 = lo_pair(make_float2(f[2], f[3]), sf, bf, h1);
}

template <typename AT>
__device__ __forceinline__ uint32_t splat(AT v) {
  const uint16_t u = *reinterpret_cast<const uint16_t*>(&v);
  return uint32_t(u) | (uint32_t(u) << 16);
}

// The 64 reconstructed weights of row r of a stage's packed tile (two per
// register, k ascending) and, for bfloat16, their residuals (lo_pair): the
// reconstruction of qlin_dequant, bit for bit.  Rows past N (row_ok false)
// give zeros.
template <int BITS, typename AT, int kSplit>
__device__ __forceinline__ void dequant_row(const uint8_t* wrow, int r, AT sc, AT bc, bool row_ok,
                                            uint32_t (&a)[32], uint32_t (&lo)[kSplit == 2 ? 32 : 1]) {
  const uint32_t s2 = row_ok ? splat(sc) : 0u, b2 = row_ok ? splat(bc) : 0u;
  if constexpr (kSplit == 2) {
    const float sv = row_ok ? Act<AT>::to_f32(sc) : 0.0f;
    const float bv = row_ok ? Act<AT>::to_f32(bc) : 0.0f;
    const float2 sf = make_float2(sv, sv), bf = make_float2(bv, bv);
    if constexpr (BITS == 4) {
      const int sw = (r >> 2) & 1;
      const uint4 v0 = *reinterpret_cast<const uint4*>(wrow + ((0 ^ sw) << 4));
      const uint4 v1 = *reinterpret_cast<const uint4*>(wrow + ((1 ^ sw) << 4));
      const uint32_t words[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int c = 0; c < 8; ++c)
        dequant_word4_split(words[c], s2, b2, sf, bf,
                            *reinterpret_cast<uint32_t(*)[4]>(a + 4 * c),
                            *reinterpret_cast<uint32_t(*)[4]>(lo + 4 * c));
    } else {
      const int sw = (r >> 1) & 3;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(wrow + ((c ^ sw) << 4));
        const uint32_t ws4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dequant_word8_split(ws4[e], s2, b2, sf, bf, a[8 * c + 2 * e], a[8 * c + 2 * e + 1],
                              lo[8 * c + 2 * e], lo[8 * c + 2 * e + 1]);
      }
    }
  } else if constexpr (BITS == 4) {
    // packed rows are 32 bytes in the 32-byte TMA swizzle: chunk c of row
    // r sits at chunk c ^ ((r >> 2) & 1)
    const int sw = (r >> 2) & 1;
    const uint4 v0 = *reinterpret_cast<const uint4*>(wrow + ((0 ^ sw) << 4));
    const uint4 v1 = *reinterpret_cast<const uint4*>(wrow + ((1 ^ sw) << 4));
    const uint32_t words[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 o = dequant_word4<AT>(words[c], s2, b2);
      a[4 * c] = o.x;
      a[4 * c + 1] = o.y;
      a[4 * c + 2] = o.z;
      a[4 * c + 3] = o.w;
    }
  } else {
    // packed rows are 64 bytes in the 64-byte TMA swizzle: chunk c of row
    // r sits at chunk c ^ ((r >> 1) & 3)
    const int sw = (r >> 1) & 3;
    uint32_t words[16];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = *reinterpret_cast<const uint4*>(wrow + ((c ^ sw) << 4));
      words[4 * c] = v.x;
      words[4 * c + 1] = v.y;
      words[4 * c + 2] = v.z;
      words[4 * c + 3] = v.w;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      dequant_word8<AT>(words[2 * c], s2, b2, a[4 * c], a[4 * c + 1]);
      dequant_word8<AT>(words[2 * c + 1], s2, b2, a[4 * c + 2], a[4 * c + 3]);
    }
  }
}

// ------------------------------------------------------------------- host
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

qlin_status make_map(CUtensorMap* map, CUtensorMapDataType dt, const void* ptr, uint64_t inner,
                     uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                     CUtensorMapSwizzle swz) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(QLIN_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, dt, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(QLIN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return QLIN_OK;
}

}  // namespace
}  // namespace qlin
