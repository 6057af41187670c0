// Public C entry points of routing and the experts' products: argument validation,
// then dispatch to the launchers.  Nothing is launched unless every check passes.

#include <cmath>

#include "qlin_internal.h"
#include "qlin_testing.h"

namespace qlin {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxPairs = int64_t(1) << 30;

qlin_status check_flags(const char* name, unsigned flags) {
  if (flags & ~unsigned(QLIN_OVERLAP_PREVIOUS))
    return fail(QLIN_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  return QLIN_OK;
}

// tokens, experts a token and experts
qlin_status check_routing(const char* name, int64_t T, int top_k, int E) {
  if (T < 0 || top_k < 1 || E < 1 || top_k > E)
    return fail(QLIN_ERR_INVALID_ARG, "%s: T=%lld top_k=%d E=%d", name, (long long)T, top_k, E);
  if (E > 512 || top_k > 32)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: E=%d (at most 512), top_k=%d (at most 32)", name, E,
                top_k);
  if (T > kMaxPairs / top_k) return fail(QLIN_ERR_UNSUPPORTED, "%s: T too large", name);
  return QLIN_OK;
}

// What qlin_expert_linear takes (with no pairs, whatever the pointers).
qlin_status check_expert_linear(const char* name, const ExpertArgs& a, int bits, int group_size,
                                qlin_dtype dtype, qlin_dtype y_dtype, size_t workspace_bytes,
                                unsigned flags) {
  qlin_status s = check_flags(name, flags);
  if (s != QLIN_OK) return s;
  if (bits != 4 && bits != 8)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: bits=%d (supported: 4, 8)", name, bits);
  if (group_size != kGroup)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: group_size=%d (supported: 64)", name, group_size);
  if (dtype != QLIN_F16 && dtype != QLIN_BF16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: dtype %d (supported: QLIN_F16, QLIN_BF16)", name,
                int(dtype));
  if (y_dtype != dtype && y_dtype != QLIN_F32)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: y dtype %d must be float32 or the activation dtype",
                name, int(y_dtype));
  if (a.n_pairs < 0 || a.pairs_per_row < 1 || a.n_pairs % a.pairs_per_row || a.E < 1 || a.N < 1 ||
      a.K < 1 || a.K % kGroup)
    return fail(QLIN_ERR_INVALID_ARG,
                "%s: n_pairs=%lld pairs_per_row=%d E=%d N=%lld K=%lld (K a multiple of %d)", name,
                (long long)a.n_pairs, a.pairs_per_row, a.E, (long long)a.N, (long long)a.K, kGroup);
  if (a.E > 512 || a.n_pairs > kMaxPairs || a.N > (int64_t(1) << 20) || a.K > 65536 ||
      int64_t(a.E) * a.N > (int64_t(1) << 30))
    return fail(QLIN_ERR_UNSUPPORTED, "%s: sizes beyond the supported range", name);
  if (a.n_pairs == 0) return QLIN_OK;
  if (!a.x || !a.order || !a.offsets || !a.wq || !a.scales || !a.biases || !a.y)
    return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (a.x_stride < a.K)
    return fail(QLIN_ERR_INVALID_ARG, "%s: x_stride is shorter than K", name);
  const size_t need = expert_linear_workspace_size(a.n_pairs, a.E, a.N, a.K);
  if (need && (!a.workspace || workspace_bytes < need))
    return fail(QLIN_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", name, need);
  if (!aligned(a.x, 16) || a.x_stride % 8 || !aligned(a.wq, 16) || !aligned(a.workspace, 16) ||
      !aligned(a.scales, 2) || !aligned(a.biases, 2) || !aligned(a.y, a.y_f32 ? 4 : 2) ||
      !aligned(a.order, 4) || !aligned(a.offsets, 4))
    return fail(QLIN_ERR_MISALIGNED,
                "%s: x, wq and workspace must be 16-byte aligned, x_stride a multiple of 8, the "
                "rest aligned to its elements", name);
  return QLIN_OK;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

size_t qlin_route_experts_workspace_size(int64_t T, int E) {
  return T < 0 || E < 1 || E > 512 ? 0 : route_experts_workspace_size(T, E);
}

qlin_status qlin_route_experts(const void* logits, int64_t logits_stride, const float* bias,
                               int scoring, int groups, int top_groups, int group_score, int top_k,
                               int renormalise, float scale, int32_t* experts, float* weights,
                               int32_t* order, int32_t* offsets, int64_t T, int E,
                               qlin_dtype ldtype, void* workspace, size_t workspace_bytes,
                               unsigned flags, void* stream) {
  const char* name = "qlin_route_experts";
  clear_error();
  qlin_status s = check_flags(name, flags);
  if (s != QLIN_OK) return s;
  if ((s = check_routing(name, T, top_k, E)) != QLIN_OK) return s;
  if (ldtype != QLIN_F32 && ldtype != QLIN_F16 && ldtype != QLIN_BF16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: logits dtype %d", name, int(ldtype));
  if ((scoring != QLIN_SOFTMAX && scoring != QLIN_SIGMOID) ||
      (group_score != QLIN_GROUP_MAX && group_score != QLIN_GROUP_TOP2) ||
      (renormalise != 0 && renormalise != 1))
    return fail(QLIN_ERR_INVALID_ARG, "%s: scoring=%d group_score=%d renormalise=%d", name, scoring,
                group_score, renormalise);
  if (groups < 1 || E % groups || top_groups < 1 || top_groups > groups)
    return fail(QLIN_ERR_INVALID_ARG, "%s: groups=%d must divide E=%d, and top_groups=%d be 1 .. groups",
                name, groups, E, top_groups);
  if (groups > 32) return fail(QLIN_ERR_UNSUPPORTED, "%s: groups=%d (at most 32)", name, groups);
  if (!std::isfinite(scale)) return fail(QLIN_ERR_INVALID_ARG, "%s: scale is not finite", name);
  if (!offsets || (T && (!logits || !experts || !weights || !order)))
    return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (logits_stride < E)
    return fail(QLIN_ERR_INVALID_ARG, "%s: logits_stride is shorter than E", name);
  const size_t need = route_experts_workspace_size(T, E);
  if (need && (!workspace || workspace_bytes < need))
    return fail(QLIN_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", name, need);
  if (!aligned(logits, ldtype == QLIN_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(experts, 4) ||
      !aligned(weights, 4) || !aligned(order, 4) || !aligned(offsets, 4) || !aligned(workspace, 16))
    return fail(QLIN_ERR_MISALIGNED,
                "%s: a pointer is not aligned to its elements, or workspace to 16 bytes", name);
  const RouteArgs a = {logits,  logits_stride, bias,        scoring, groups, top_groups,
                       group_score, top_k,     renormalise, scale,   experts, weights,
                       order,   offsets,       T,           E,       ldtype};
  return launch_route_experts(a, workspace, flags, reinterpret_cast<cudaStream_t>(stream));
}

size_t qlin_expert_linear_workspace_size(int64_t n_pairs, int E, int64_t N, int64_t K) {
  return n_pairs < 1 || E < 1 || N < 1 || K < 1 ? 0 : expert_linear_workspace_size(n_pairs, E, N, K);
}

qlin_status qlin_expert_linear(const void* x, int64_t x_stride, int pairs_per_row,
                               const int32_t* order, const int32_t* offsets, int64_t n_pairs,
                               const uint32_t* wq, const void* scales, const void* biases, void* y,
                               int E, int64_t N, int64_t K, int bits, int group_size,
                               qlin_dtype dtype, qlin_dtype y_dtype, void* workspace,
                               size_t workspace_bytes, unsigned flags, void* stream) {
  const ExpertArgs a = {x,       x_stride, pairs_per_row, order,  offsets,
                        n_pairs, wq,       scales,        biases, y,
                        y_dtype == QLIN_F32 ? 1 : 0, E, N, K, workspace};
  clear_error();
  const qlin_status s = check_expert_linear("qlin_expert_linear", a, bits, group_size, dtype,
                                            y_dtype, workspace_bytes, flags);
  if (s != QLIN_OK || n_pairs == 0) return s;
  return launch_expert_linear(a, bits, dtype, flags, reinterpret_cast<cudaStream_t>(stream));
}

qlin_status qlin_testing_expert_linear_stalled(
    const void* x, int64_t x_stride, int pairs_per_row, const int32_t* order,
    const int32_t* offsets, int64_t n_pairs, const uint32_t* wq, const void* scales,
    const void* biases, void* y, int E, int64_t N, int64_t K, void* workspace,
    size_t workspace_bytes, int stalled_stage, unsigned wait_limit_us, void* stream) {
  const char* name = "qlin_testing_expert_linear_stalled";
  const ExpertArgs a = {x,  x_stride, pairs_per_row, order, offsets, n_pairs, wq,       scales,
                        biases, y,    0,             E,     N,       K,       workspace};
  clear_error();
  const qlin_status s = check_expert_linear(name, a, 4, kGroup, QLIN_F16, QLIN_F16,
                                            workspace_bytes, 0);
  if (s != QLIN_OK) return s;
  if (stalled_stage < 0 || wait_limit_us < 1000 || wait_limit_us > 2000000)
    return fail(QLIN_ERR_INVALID_ARG, "%s: stalled_stage=%d wait_limit_us=%u (1000 .. 2000000)",
                name, stalled_stage, wait_limit_us);
  if (expert_linear_workspace_size(n_pairs, E, N, K) == 0)
    return fail(QLIN_ERR_INVALID_ARG, "%s: a call that waits for nothing", name);
  return launch_expert_stalled(a, stalled_stage, wait_limit_us,
                               reinterpret_cast<cudaStream_t>(stream));
}

qlin_status qlin_combine_experts(const void* y, const int32_t* experts, const float* weights,
                                 const void* add, int64_t add_stride, void* out, int64_t T,
                                 int top_k, int64_t N, qlin_dtype dtype, qlin_dtype y_dtype,
                                 unsigned flags, void* stream) {
  const char* name = "qlin_combine_experts";
  clear_error();
  qlin_status s = check_flags(name, flags);
  if (s != QLIN_OK) return s;
  if (dtype != QLIN_F16 && dtype != QLIN_BF16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: dtype %d (supported: QLIN_F16, QLIN_BF16)", name,
                int(dtype));
  if (y_dtype != dtype && y_dtype != QLIN_F32)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: y dtype %d must be float32 or the activation dtype",
                name, int(y_dtype));
  if (T < 0 || top_k < 1 || N < 1)
    return fail(QLIN_ERR_INVALID_ARG, "%s: T=%lld top_k=%d N=%lld", name, (long long)T, top_k,
                (long long)N);
  if (top_k > 32 || T > kMaxPairs / top_k || N > (int64_t(1) << 20))
    return fail(QLIN_ERR_UNSUPPORTED, "%s: sizes beyond the supported range", name);
  if (T == 0) return QLIN_OK;
  if (!y || !experts || !weights || !out)
    return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (add && add_stride < N)
    return fail(QLIN_ERR_INVALID_ARG, "%s: add_stride is shorter than N", name);
  if (!aligned(y, y_dtype == QLIN_F32 ? 4 : 2) || !aligned(add, 2) || !aligned(out, 2) ||
      !aligned(experts, 4) || !aligned(weights, 4))
    return fail(QLIN_ERR_MISALIGNED, "%s: a pointer is not aligned to its elements", name);
  return launch_combine_experts(y, experts, weights, add, add ? add_stride : 0, out, T, top_k, N,
                                dtype, y_dtype, flags, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
