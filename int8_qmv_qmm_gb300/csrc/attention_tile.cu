// Attention of slots with many new rows (prompts and their chunks).
//
// One CTA for each 16 rows and key/value head.  Its warps take the blocks in
// turn, each with a running maximum and sum of its own (m16n8k16 products), and
// are joined at the end.

#include "attention_core.cuh"

namespace qlin {
namespace attention {

__device__ unsigned int g_tile_status = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;

__device__ __forceinline__ void report(unsigned bit) { atomicOr(&g_tile_status, bit); }

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) tile_kernel(const Args a) {
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
        const int64_t rows = int64_t(r.n) * a.group;
        return rows > kSplitRows ? (rows + kRows - 1) / kRows : 0;
      }))
    return;
  const SlotRows r = slot_rows(a.starts, a.c.lens, b, a.n_tokens);
  const int rows = r.n * a.group, r0 = int(tile) * kRows;
  const bool over = r.n > a.max_new;  // (the split kernel reports it)
  Warp<T, D, 2> w;
  w.init();
  const T* qp[2];
  int pos[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int row = r0 + 8 * n + g;
    qp[n] = row < rows ? static_cast<const T*>(a.q) + (r.row0 + row / a.group) * a.q_stride +
                             (kvh * a.group + row % a.group) * D
                       : nullptr;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int mine = r0 + 8 * n + 2 * t + i;
      pos[n][i] = mine < rows ? r.held + mine / a.group : -1;
    }
  }
  w.load_q(qp, lane);
  w.prepare_q(a.scale_log2, lane);
  const int total = r.held + r.n, full = total / kBlock;
  const int last = r.held + (min(r0 + kRows, rows) - 1) / a.group;  // last position seen
  const int first = r.held + r0 / a.group;
  if (!over) {
    for (int j = warp; j <= last / kBlock; j += kWarps) {
      int seen[2][2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
        seen[n][0] = pos[n][0] - j * kBlock + 1, seen[n][1] = pos[n][1] - j * kBlock + 1;
      if (j < full) {
        const int64_t page = page_of(a.c, b, j);
        if (page < 0) {
          if (lane == 0) report(kStatusPage);
          continue;
        }
        const int64_t at = page * a.c.kv_heads + kvh;
        const uint8_t* codes = static_cast<const uint8_t*>(a.c.pages) + at * 2 * kBlock * D;
        float s[4][2][4];
        uint32_t p[4][2][2];
        w.scores(codes, s, lane);
        w.probabilities(s, p, a.c.scales[2 * at], a.c.scales[2 * at + 1], seen,
                        first < j * kBlock + kBlock - 1, lane);
        w.values(codes + kBlock * D, p, lane);
      } else {
        w.tail(static_cast<const T*>(a.c.tail) +
                   (int64_t(b) * a.c.kv_heads + kvh) * 2 * kBlock * D,
               total - j * kBlock, qp, a.scale_log2, seen, lane);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 8 * n + 2 * t + i;
      float l = w.l[n][i];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) {
        s_m[warp][row] = w.m[n][i];
        s_l[warp][row] = l;
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        s_o[warp][row][16 * c + g] = w.o[c][n][i] * w.unit;
        s_o[warp][row][16 * c + 8 + g] = w.o[c][n][2 + i] * w.unit;
      }
    }
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
  cudaLaunchKernelEx(&cfg, tile_kernel<T, D>, a);
}

}  // namespace

void launch_tile(const Args& a, unsigned flags, cudaStream_t st) {
  if (a.c.dtype == QLIN_F16)
    a.c.head_dim == 64 ? launch_t<__half, 64>(a, flags, st) : launch_t<__half, 128>(a, flags, st);
  else
    a.c.head_dim == 64 ? launch_t<__nv_bfloat16, 64>(a, flags, st)
                       : launch_t<__nv_bfloat16, 128>(a, flags, st);
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
