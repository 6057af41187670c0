// The parts that the split kernel leaves in the workspace, and how they are joined:
// by a kernel of its own, or beside the tile kernel's pieces.
#pragma once

#include <algorithm>

#include "attention_core.cuh"

namespace qlin {
namespace attention {

constexpr int kSplitWarps = 8;        // of a CTA
constexpr int kSplitTile = 8;         // rows of a tile
constexpr int kSplitMaxWarps = 2048;  // of the grid
constexpr int kJoinThreads = 512;
constexpr int kSplitJoinPerSm = 2;

// A tile whose blocks begin in warp i's share and pass its end: warps i .. last
// have parts.
struct alignas(16) Split {
  int last;      // -1: warp i has none
  int token0;    // first row of the slot in q and out
  int row0;      // of the tile in the slot
  int kvh_here;  // 16 * key/value head + rows of the tile
};

// A part: sums [D][8 rows], then the rows' m and l.
template <int D>
constexpr int kSplitPart = kSplitTile * (D + 2);  // floats

// Scratch of the split kernel: two parts for each of its warps.
struct SplitScratch {
  Split* splits;
  float* parts;
  int warps;
};
inline SplitScratch split_scratch(void* workspace, int sms) {
  const int warps = std::min(sms, kSplitMaxWarps / kSplitWarps) * kSplitWarps;
  Split* splits = static_cast<Split*>(workspace);
  return SplitScratch{splits, reinterpret_cast<float*>(splits + warps), warps};
}

// Joins the parts of the tiles that pass the end of a warp's share.  Each CTA
// lists them (the order is that of the warps).  A team of warps takes a slice, 16
// dimensions of a tile's 8 rows: its warps (4 rows of one dimension a thread) take
// a part each in turn, and are added up in order.  Teams are a whole CTA where the
// slices are no more than the CTAs (few, long lists of parts), else four warps.
// (Whole CTAs alone: 52.8 us for 32 sequences of 8192 tokens with the split kernel,
// 32.8 for 36 rows of 3000; with both sizes 49.2 and 29.4.  A warp for each slice of
// up to 8 parts: 49.7 and 33.2, but 16 sequences of mixed lengths 62 for 59.)
//
// The CTA is `block` of `blocks`, all of kJoinThreads threads.
template <typename T, int D>
__device__ void join_split(const Args& a, const SplitScratch& sc, int block, int blocks) {
  const float* parts = sc.parts;
  const Split* splits = sc.splits;
  constexpr int kSlices = D / 16, kGroups = kJoinThreads / 32;
  constexpr int kRounds = kSplitMaxWarps / kJoinThreads;
  __shared__ int s_which[kSplitMaxWarps], s_count[kRounds][kGroups];
  __shared__ float4 s_o[kGroups][32], s_m[kGroups][2], s_l[kGroups][2];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  unsigned ballot[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int w = i * kJoinThreads + threadIdx.x;
    ballot[i] = w < sc.warps && __ldcg(&splits[w].last) >= 0;
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    ballot[i] = __ballot_sync(0xffffffffu, ballot[i]);
    if (lane == 0) s_count[i][group] = __popc(ballot[i]);
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    int at = n;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      if (k < group) at += s_count[i][k];
      n += s_count[i][k];
    }
    if (ballot[i] >> lane & 1)
      s_which[at + __popc(ballot[i] & ((1u << lane) - 1))] = i * kJoinThreads + int(threadIdx.x);
  }
  __syncthreads();
  const int size = n * kSlices <= blocks ? kGroups : 4, teams = kGroups / size;
  const int team = group / size, g0 = team * size;  // and the team's first warp
  auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * size) : "memory"); };
  for (int task = block * teams + team; task < n * kSlices; task += blocks * teams) {
    const int first = s_which[task / kSlices], d0 = task % kSlices * 16;
    const Split sp = splits[first];
    // this thread: dimension d0 + lane/2, rows 4 * (lane%2) ..
    const int d = d0 + (lane >> 1), half = lane & 1;
    float m[4], l[4], o[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) m[r] = -INFINITY, l[r] = o[r] = 0.f;
#pragma unroll 4
    for (int k = first + group - g0; k <= sp.last; k += size) {
      const float* part = parts + size_t(2 * k + (k == first ? 1 : 0)) * kSplitPart<D>;
      const float4 pm = __ldcg(reinterpret_cast<const float4*>(part + kSplitTile * D) + half);
      const float4 pl = __ldcg(reinterpret_cast<const float4*>(part + kSplitTile * (D + 1)) + half);
      const float4 po = __ldcg(reinterpret_cast<const float4*>(part + kSplitTile * d) + half);
      const float vm[4] = {pm.x, pm.y, pm.z, pm.w}, vl[4] = {pl.x, pl.y, pl.z, pl.w},
                  vo[4] = {po.x, po.y, po.z, po.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float next = fmaxf(m[r], vm[r]), base = next == -INFINITY ? 0.f : next;
        const float f0 = exp2_fast(m[r] - base), f1 = exp2_fast(vm[r] - base);
        l[r] = l[r] * f0 + vl[r] * f1;
        o[r] = o[r] * f0 + vo[r] * f1;
        m[r] = next;
      }
    }
    s_o[group][lane] = make_float4(o[0], o[1], o[2], o[3]);
    if (lane < 2) {
      s_m[group][lane] = make_float4(m[0], m[1], m[2], m[3]);
      s_l[group][lane] = make_float4(l[0], l[1], l[2], l[3]);
    }
    meet();
    // 128 sums: thread i of the team takes row i/16, dimension d0 + i%16
    const int i = threadIdx.x - 32 * g0, row = i >> 4, dd = i & 15, here = sp.kvh_here & 15;
    if (row < here) {
      auto value = [&](const float4* v) { return reinterpret_cast<const float*>(v)[row & 3]; };
      float top = -INFINITY, sum = 0.f, out = 0.f;
#pragma unroll 4
      for (int k = g0; k < g0 + size; ++k) top = fmaxf(top, value(&s_m[k][row >> 2]));
#pragma unroll 4
      for (int k = g0; k < g0 + size; ++k) {
        const float vm = value(&s_m[k][row >> 2]);
        const float f = vm == -INFINITY ? 0.f : exp2_fast(vm - top);
        sum += value(&s_l[k][row >> 2]) * f;
        out += value(&s_o[k][2 * dd + (row >> 2)]) * f;
      }
      const int rr = sp.row0 + row, kvh = sp.kvh_here >> 4;
      static_cast<T*>(a.out)[(int64_t(sp.token0 + rr / a.group) * a.q_heads + kvh * a.group +
                              rr % a.group) *
                                 D +
                             d0 + dd] = Act<T>::from_f32_rn(out * share_of(sum));
    }
    meet();
  }
}

}  // namespace attention
}  // namespace qlin
