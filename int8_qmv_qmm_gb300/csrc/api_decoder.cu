// Public C entry points of what stands between a decoder's linears: argument
// validation, then dispatch to the launchers.  Nothing is launched unless
// every check passes.

#include <cmath>

#include "qlin_internal.h"
#include "qlin_testing.h"

namespace qlin {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxRows = int64_t(1) << 30;

qlin_status check_flags(const char* name, unsigned flags) {
  if (flags & ~unsigned(QLIN_OVERLAP_PREVIOUS))
    return fail(QLIN_ERR_INVALID_ARG, "%s: unknown flags 0x%x", name, flags);
  return QLIN_OK;
}

qlin_status check_cache(const char* name, const qlin_kv_cache* c) {
  if (!c) return fail(QLIN_ERR_INVALID_ARG, "%s: null cache", name);
  if (c->dtype != QLIN_F16 && c->dtype != QLIN_BF16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: cache dtype %d (supported: QLIN_F16, QLIN_BF16)", name,
                int(c->dtype));
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: head_dim=%d (supported: 64, 128)", name, c->head_dim);
  if (c->slots < 1 || c->kv_heads < 1 || c->max_blocks < 1 || c->n_pages < 1)
    return fail(QLIN_ERR_INVALID_ARG,
                "%s: slots, kv_heads, max_blocks and n_pages must be positive", name);
  if (c->kv_heads > 65535 || c->slots > 1024 || c->n_pages > (int64_t(1) << 31))
    return fail(QLIN_ERR_UNSUPPORTED, "%s: cache beyond the supported range", name);
  if (!c->pages || !c->scales || !c->tail || !c->table || !c->lens)
    return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer in the cache", name);
  if (!aligned(c->pages, 16) || !aligned(c->tail, 16) || !aligned(c->scales, 8) ||
      !aligned(c->table, 4) || !aligned(c->lens, 4))
    return fail(QLIN_ERR_MISALIGNED,
                "%s: pages and tail must be 16-byte aligned, scales 8, table and lens 4", name);
  return QLIN_OK;
}

qlin_status check_rows(const char* name, const qlin_kv_cache* c, int64_t n_tokens, int q_heads) {
  if (n_tokens < 0) return fail(QLIN_ERR_INVALID_ARG, "%s: n_tokens=%lld", name, (long long)n_tokens);
  if (q_heads < 1 || q_heads % c->kv_heads)
    return fail(QLIN_ERR_INVALID_ARG, "%s: q_heads=%d must be a positive multiple of kv_heads=%d",
                name, q_heads, c->kv_heads);
  if (q_heads / c->kv_heads > 16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: more than 16 query heads to a key/value head", name);
  if (n_tokens > kMaxRows || n_tokens * q_heads > kMaxRows)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: n_tokens=%lld too large", name, (long long)n_tokens);
  return QLIN_OK;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_add_rms_norm(const void* x, int64_t x_stride, const void* weight,
                              const void* residual, int64_t residual_stride, void* residual_out,
                              void* y, int64_t M, int64_t K, float eps, qlin_dtype dtype,
                              qlin_dtype rdtype, unsigned flags, void* stream) {
  const char* name = "qlin_add_rms_norm";
  clear_error();
  qlin_status s = check_flags(name, flags);
  if (s != QLIN_OK) return s;
  if (dtype != QLIN_F16 && dtype != QLIN_BF16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: dtype %d (supported: QLIN_F16, QLIN_BF16)", name,
                int(dtype));
  if (rdtype != dtype && rdtype != QLIN_F32)
    return fail(QLIN_ERR_UNSUPPORTED,
                "%s: residual dtype %d must be float32 or the activation dtype", name,
                int(rdtype));
  if (M < 0 || K < 1) return fail(QLIN_ERR_INVALID_ARG, "%s: M=%lld K=%lld", name, (long long)M, (long long)K);
  if (K > 32768) return fail(QLIN_ERR_UNSUPPORTED, "%s: K=%lld (at most 32768)", name, (long long)K);
  if (M > kMaxRows) return fail(QLIN_ERR_UNSUPPORTED, "%s: M too large", name);
  if (!(eps >= 0.f)) return fail(QLIN_ERR_INVALID_ARG, "%s: eps must not be negative", name);
  if (M == 0) return QLIN_OK;
  if (!x || !weight || !y) return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (residual_out && !residual)
    return fail(QLIN_ERR_INVALID_ARG, "%s: residual_out without a residual", name);
  if (x_stride < K || (residual && residual_stride < K))
    return fail(QLIN_ERR_INVALID_ARG, "%s: a row stride is shorter than K", name);
  const uintptr_t ra = rdtype == QLIN_F32 ? 4 : 2;
  if (!aligned(x, 2) || !aligned(weight, 2) || !aligned(y, 2) || !aligned(residual, ra) ||
      !aligned(residual_out, ra))
    return fail(QLIN_ERR_MISALIGNED, "%s: a pointer is not aligned to its elements", name);
  return launch_add_rms_norm(x, x_stride, weight, residual, residual ? residual_stride : 0,
                             residual_out, y, M, K, eps, dtype, rdtype, flags,
                             reinterpret_cast<cudaStream_t>(stream));
}

qlin_status qlin_rope_table(float* table, int64_t n_positions, int rot_dim, double base,
                            double factor, double short_wavelength, double long_wavelength,
                            void* stream) {
  const char* name = "qlin_rope_table";
  clear_error();
  if (n_positions < 0 || rot_dim < 2 || rot_dim % 2)
    return fail(QLIN_ERR_INVALID_ARG, "%s: n_positions=%lld rot_dim=%d", name,
                (long long)n_positions, rot_dim);
  if (!(base > 1.0) || !(factor >= 1.0) || !(short_wavelength >= 0.0) ||
      !(long_wavelength >= short_wavelength) || !std::isfinite(base) || !std::isfinite(factor) ||
      !std::isfinite(long_wavelength))
    return fail(QLIN_ERR_INVALID_ARG, "%s: base, factor or wavelengths out of range", name);
  if (rot_dim > 1024 || n_positions > (int64_t(1) << 24))
    return fail(QLIN_ERR_UNSUPPORTED, "%s: table beyond the supported range", name);
  if (n_positions == 0) return QLIN_OK;
  if (!table) return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned(table, 8)) return fail(QLIN_ERR_MISALIGNED, "%s: table must be 8-byte aligned", name);
  return launch_rope_table(table, n_positions, rot_dim, base, factor, short_wavelength,
                           long_wavelength, reinterpret_cast<cudaStream_t>(stream));
}

qlin_status qlin_rope_append(const void* qkv, int64_t qkv_stride, void* q_out,
                             const float* table, int64_t n_positions, int rot_dim,
                             int interleaved, const qlin_kv_cache* cache, const int32_t* starts,
                             int64_t n_tokens, int q_heads, unsigned flags, void* stream) {
  const char* name = "qlin_rope_append";
  clear_error();
  qlin_status s = check_flags(name, flags);
  if (s != QLIN_OK) return s;
  if ((s = check_cache(name, cache)) != QLIN_OK) return s;
  if ((s = check_rows(name, cache, n_tokens, q_heads)) != QLIN_OK) return s;
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: rot_dim=%d (a multiple of 16, at most head_dim=%d)",
                name, rot_dim, cache->head_dim);
  if (interleaved != 0 && interleaved != 1)
    return fail(QLIN_ERR_INVALID_ARG, "%s: interleaved=%d (0 or 1)", name, interleaved);
  if (n_positions < 0) return fail(QLIN_ERR_INVALID_ARG, "%s: n_positions < 0", name);
  if (n_tokens == 0) return QLIN_OK;
  if (!qkv || !q_out || !starts || (rot_dim && !table))
    return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (qkv_stride < int64_t(q_heads + 2 * cache->kv_heads) * cache->head_dim)
    return fail(QLIN_ERR_INVALID_ARG, "%s: qkv_stride is shorter than a row", name);
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || qkv_stride % 8 || !aligned(table, 16) ||
      !aligned(starts, 4))
    return fail(QLIN_ERR_MISALIGNED,
                "%s: qkv, q_out and table must be 16-byte aligned, qkv_stride a multiple of 8",
                name);
  return launch_rope_append(qkv, qkv_stride, q_out, table, n_positions, rot_dim, interleaved,
                            *cache, starts, n_tokens, q_heads, flags,
                            reinterpret_cast<cudaStream_t>(stream));
}

qlin_status qlin_cache_dequant(const qlin_kv_cache* cache, const int32_t* page_ids, int64_t n,
                               void* out, void* stream) {
  const char* name = "qlin_cache_dequant";
  clear_error();
  qlin_status s = check_cache(name, cache);
  if (s != QLIN_OK) return s;
  if (n < 0) return fail(QLIN_ERR_INVALID_ARG, "%s: n=%lld", name, (long long)n);
  if (n == 0) return QLIN_OK;
  if (!page_ids || !out) return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned(out, 16) || !aligned(page_ids, 4))
    return fail(QLIN_ERR_MISALIGNED, "%s: out must be 16-byte aligned", name);
  return launch_cache_dequant(*cache, page_ids, n, out, reinterpret_cast<cudaStream_t>(stream));
}

size_t qlin_cache_attention_workspace_size(int head_dim) {
  return cache_attention_workspace_size(head_dim);
}

qlin_status qlin_cache_attention(const void* q, int64_t q_stride, void* out,
                                 const qlin_kv_cache* cache, const int32_t* starts,
                                 int64_t n_tokens, int q_heads, float scale, int max_new,
                                 void* workspace, size_t workspace_bytes, unsigned flags,
                                 void* stream) {
  const char* name = "qlin_cache_attention";
  clear_error();
  qlin_status s = check_flags(name, flags);
  if (s != QLIN_OK) return s;
  if ((s = check_cache(name, cache)) != QLIN_OK) return s;
  if ((s = check_rows(name, cache, n_tokens, q_heads)) != QLIN_OK) return s;
  if (!std::isfinite(scale)) return fail(QLIN_ERR_INVALID_ARG, "%s: scale is not finite", name);
  if (max_new < 0) return fail(QLIN_ERR_INVALID_ARG, "%s: max_new=%d", name, max_new);
  if (n_tokens == 0) return QLIN_OK;
  if (!q || !out || !starts) return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (q_stride < int64_t(q_heads) * cache->head_dim)
    return fail(QLIN_ERR_INVALID_ARG, "%s: q_stride is shorter than a row", name);
  const size_t need = cache_attention_workspace_size(cache->head_dim);
  if (!workspace || workspace_bytes < need)
    return fail(QLIN_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", name, need);
  if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || !aligned(workspace, 16) ||
      !aligned(starts, 4))
    return fail(QLIN_ERR_MISALIGNED,
                "%s: q, out and workspace must be 16-byte aligned, q_stride a multiple of 8",
                name);
  return launch_cache_attention(q, q_stride, out, *cache, starts, n_tokens, q_heads, scale,
                                max_new, workspace, flags,
                                reinterpret_cast<cudaStream_t>(stream));
}

qlin_status qlin_sample(const void* logits, int64_t logits_stride, const float* u,
                        const float* temperature, const int32_t* top_k, const float* top_p,
                        const float* min_p, int32_t* tokens, float* probs, int64_t M, int64_t V,
                        qlin_dtype ldtype, unsigned flags, void* stream) {
  const char* name = "qlin_sample";
  clear_error();
  qlin_status s = check_flags(name, flags);
  if (s != QLIN_OK) return s;
  if (ldtype != QLIN_F32 && ldtype != QLIN_F16 && ldtype != QLIN_BF16)
    return fail(QLIN_ERR_UNSUPPORTED, "%s: logits dtype %d", name, int(ldtype));
  if (M < 0 || V < 1) return fail(QLIN_ERR_INVALID_ARG, "%s: M=%lld V=%lld", name, (long long)M, (long long)V);
  if (V > 262144) return fail(QLIN_ERR_UNSUPPORTED, "%s: V=%lld (at most 262144)", name, (long long)V);
  if (M > kMaxRows) return fail(QLIN_ERR_UNSUPPORTED, "%s: M too large", name);
  if (M == 0) return QLIN_OK;
  if (!logits || !u || !temperature || !top_k || !top_p || !min_p || !tokens)
    return fail(QLIN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (logits_stride < V)
    return fail(QLIN_ERR_INVALID_ARG, "%s: logits_stride is shorter than V", name);
  if (!aligned(logits, ldtype == QLIN_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) ||
      !aligned(probs, 4))
    return fail(QLIN_ERR_MISALIGNED, "%s: a pointer is not aligned to its elements", name);
  return launch_sample(logits, logits_stride, u, temperature, top_k, top_p, min_p, tokens, probs,
                       M, V, ldtype, flags, reinterpret_cast<cudaStream_t>(stream));
}

qlin_status qlin_testing_sample_plan(int64_t M, int64_t V, int sm_count, int* ranks, int* part,
                                     int* limb_bits) {
  clear_error();
  if (M < 1 || V < 1 || V > 262144 || sm_count < 1 || !ranks || !part || !limb_bits)
    return fail(QLIN_ERR_INVALID_ARG, "qlin_testing_sample_plan: M=%lld V=%lld sm_count=%d",
                (long long)M, (long long)V, sm_count);
  const SamplePlan p = sample_plan(M, V, sm_count);
  *ranks = p.ranks;
  *part = p.part;
  *limb_bits = p.limb;
  return QLIN_OK;
}

qlin_status qlin_testing_sample_quotient(const float* a, const float* tau, float* q, int64_t n) {
  clear_error();
  if (n < 0 || (n && (!a || !tau || !q)))
    return fail(QLIN_ERR_INVALID_ARG, "qlin_testing_sample_quotient: n=%lld", (long long)n);
  for (int64_t i = 0; i < n; ++i) q[i] = sample_quotient(a[i], tau[i]);
  return QLIN_OK;
}

}  // extern "C"
