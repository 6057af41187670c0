// What the cache kernels share: the cache as the kernels see it, the rows of a
// slot, and the status bits of what they refuse.
#pragma once

#include <stdint.h>

#include "device_common.cuh"
#include "qlin_internal.h"

namespace qlin {

constexpr int kBlock = QLIN_KV_BLOCK;

// Bits of the cache kernels' status words (qlin_device_status shifts them by 24).
enum : unsigned {
  kStatusRows = 1u,      // rows outside n_tokens, or a negative length
  kStatusPage = 2u,      // a page outside n_pages, or a slot past max_blocks
  kStatusPosition = 4u,  // a position outside the table
  kStatusMaxNew = 8u,    // a slot with more than max_new rows
  kStatusWait = 16u,     // a wait that gave up
};

// The rows of the call that slot b owns, and the tokens it held before.
struct SlotRows {
  int64_t row0;
  int n;
  int held;
  bool bad;  // the arrays are not what the call says: the slot is left out
};

__device__ __forceinline__ SlotRows slot_rows(const int32_t* __restrict__ starts,
                                              const int32_t* __restrict__ lens, int b,
                                              int64_t n_tokens) {
  const int64_t s0 = starts[b], s1 = starts[b + 1];
  const int64_t held = lens[b];
  SlotRows r;
  r.row0 = s0;
  r.bad = s0 < 0 || s1 < s0 || s1 > n_tokens || held < 0 || held + (s1 - s0) > 0x7fffffff;
  r.n = r.bad ? 0 : static_cast<int>(s1 - s0);
  r.held = r.bad ? 0 : static_cast<int>(held);
  return r;
}

// The page of block j of slot b, or -1 where there is none.
__device__ __forceinline__ int64_t page_of(const qlin_kv_cache& c, int b, int j) {
  if (j >= c.max_blocks) return -1;
  const int64_t p = c.table[int64_t(b) * c.max_blocks + j];
  return p >= 0 && p < c.n_pages ? p : -1;
}

// Finds which slot the `item`-th unit of work belongs to, where slot b has
// count(b) units: sets b and the unit's place within the slot; false when the
// slots have fewer units.  One warp, converged; the same answer in every lane.
template <class Count>
__device__ __forceinline__ bool find_slot(int slots, int64_t item, int* slot, int64_t* place,
                                          Count count) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int b0 = 0; b0 < slots; b0 += 32) {
    const int b = b0 + lane;
    const int64_t n = b < slots ? count(b) : 0;
    int64_t upto = n;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > item);
    if (past) {
      const int l = __ffs(past) - 1;
      *slot = b0 + l;
      *place = item - before - __shfl_sync(0xffffffffu, upto - n, l);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

}  // namespace qlin
