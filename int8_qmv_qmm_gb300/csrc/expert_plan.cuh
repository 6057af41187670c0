// What the kernels of the experts' products share: the rows of an expert in a
// routing's plan, as far as the plan is what the call says.
#pragma once

#include <stdint.h>

#include "qlin_internal.h"

namespace qlin {

struct ExpertRows {
  int first;  // in order
  int n;
  bool bad;   // the offsets are not those of a plan: the expert is left out
};

__device__ __forceinline__ ExpertRows expert_rows(const ExpertArgs& a, int expert) {
  const int first = a.offsets[expert], end = a.offsets[expert + 1];
  ExpertRows r;
  r.bad = first < 0 || end < first || end > a.n_pairs;
  r.first = r.bad ? 0 : first;
  r.n = r.bad ? 0 : end - first;
  return r;
}

}  // namespace qlin
