// cache_attention: attention of new tokens over the 8-bit key/value cache
// (qlin.h has the formats).  Which kernel takes a slot goes by its rows, new
// tokens times the query heads that share a key/value head:
//   up to kSplitRows   attention_split.cu: the cache is read once, split over
//                      all SMs along its length
//   more               attention_tile.cu: products of 128 rows
// The host only knows the largest count (max_new), so with prompts among the
// slots it launches both, each for its own, and then one kernel that joins what both
// have left in parts.  Each starts while the one before it ends and waits for it
// before it reads anything: only that wait makes what came before the call visible.

#include "attention_core.cuh"

namespace qlin {

size_t cache_attention_workspace_size(int head_dim) {
  return attention::split_workspace_size(head_dim) + attention::tile_workspace_size(head_dim);
}

qlin_status launch_cache_attention(const void* q, int64_t q_stride, void* out,
                                   const qlin_kv_cache& c, const int32_t* starts,
                                   int64_t n_tokens, int q_heads, float scale, int max_new,
                                   void* workspace, unsigned flags, cudaStream_t st) {
  const attention::Args a = {q,
                             q_stride,
                             out,
                             c,
                             starts,
                             n_tokens,
                             q_heads,
                             q_heads / c.kv_heads,
                             scale * 1.4426950408889634f,
                             max_new};
  const bool tile = int64_t(max_new) * a.group > attention::kSplitRows;
  // (a kernel whose predecessor was not launched would read what it never wrote)
  cudaError_t e = attention::launch_split(a, workspace, !tile, flags, st);
  if (e == cudaSuccess && tile)
    e = attention::launch_tile(
        a, static_cast<uint8_t*>(workspace) + attention::split_workspace_size(c.head_dim),
        workspace, st);
  const qlin_status s = check_launch("qlin_cache_attention");
  return e == cudaSuccess || s != QLIN_OK
             ? s
             : fail(QLIN_ERR_CUDA, "qlin_cache_attention: %s", cudaGetErrorString(e));
}

cudaError_t attention_take_device_status(unsigned* flags) {
  unsigned s = 0, t = 0;
  cudaError_t e = attention::split_take_status(&s);
  if (e == cudaSuccess) e = attention::tile_take_status(&t);
  *flags = s | t;
  return e;
}

}  // namespace qlin
