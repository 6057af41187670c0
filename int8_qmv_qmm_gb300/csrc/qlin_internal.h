// Internal declarations shared by the libqlin translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qlin.h"

namespace qlin {

// Records a formatted detail message for qlin_last_error() and returns s.
qlin_status fail(qlin_status s, const char* fmt, ...);

// Empties the detail message (each entry point's first step).
void clear_error();

// Maps a CUDA runtime error (if any) from the last launch to a status.
qlin_status check_launch(const char* what);

// Number of SMs of the current device (cached per device).
int sm_count();

// Lets a kernel have `bytes` of dynamic shared memory on the current device; a
// repeated call costs a look at `done` (one per kernel, its bits the devices).
bool allow_shared(const void* kernel, int bytes, std::atomic<unsigned long long>* done);

// Launchers.  Arguments are already validated by the public entry points.
qlin_status launch_quantize(const float* w, int64_t N, int64_t K, int bits, qlin_dtype sdtype,
                            uint32_t* wq, void* scales, void* biases, cudaStream_t st);
qlin_status launch_dequant(const uint32_t* wq, const void* scales, const void* biases, int64_t N,
                           int64_t K, int bits, qlin_dtype sdtype, qlin_dtype out_dtype,
                           void* w_out, cudaStream_t st);
// A linear layer's epilogue: the layer bias (activation dtype [N], or null)
// added before the final rounding, and float32 output instead of the
// activation dtype.
struct Epilogue {
  const void* bias;
  int y_f32;
};

qlin_status launch_qmv(const void* x, const uint32_t* wq, const void* scales, const void* biases,
                       void* y, int64_t M, int64_t N, int64_t K, int bits, qlin_dtype dtype,
                       unsigned flags, const Epilogue& ep, cudaStream_t st);
qlin_status launch_qmm(const void* x, const uint32_t* wq, const void* scales, const void* biases,
                       void* y, int64_t M, int64_t N, int64_t K, int bits, qlin_dtype dtype,
                       unsigned flags, const Epilogue& ep, cudaStream_t st);

// Limits of the chain kernel's waits for an input link.  stalled_link >= 0
// (tests only) makes the readers of that link wait for one row block more
// than it has, so that their wait runs out.
struct ChainWaitOptions {
  unsigned long long dep_wait_ns;
  int stalled_link;
};
constexpr ChainWaitOptions kDefaultChainWaits = {2000000000ull, -1};

qlin_status launch_qmv_chain(const void* x0, const qlin_link* links, int n_links, int bits,
                             qlin_dtype dtype, void* ws, const ChainWaitOptions& wo,
                             cudaStream_t st);
int chain_max_links();

// The number of CTAs qlin_qmv gives each row block (its split of K) for an
// N x K matrix of `bits`-bit codes on a device with `sms` SMs.
int qmv_plan_split(int64_t N, int64_t K, int bits, int sms);

// ------------------------------------------- between a decoder's linears
// (add_rms_norm.cu, rope_append.cu, cache_attention.cu, sample.cu)
qlin_status launch_add_rms_norm(const void* x, int64_t x_stride, const void* weight,
                                const void* residual, int64_t residual_stride,
                                void* residual_out, void* y, int64_t M, int64_t K, float eps,
                                qlin_dtype dtype, qlin_dtype rdtype, unsigned flags,
                                cudaStream_t st);
qlin_status launch_rope_table(float* table, int64_t n_positions, int rot_dim, double base,
                              double factor, double short_wavelength, double long_wavelength,
                              cudaStream_t st);
// Norms of the queries and keys of each head before the rotation (weights
// [head_dim]; both null: none).
struct HeadNorms {
  const void* q;
  const void* k;
  float eps;
};
qlin_status launch_rope_append(const void* qkv, int64_t qkv_stride, void* q_out,
                               const float* table, int64_t n_positions, int rot_dim,
                               int interleaved, const qlin_kv_cache& c, const int32_t* starts,
                               int64_t n_tokens, int q_heads, const HeadNorms& norms,
                               unsigned flags, cudaStream_t st);
qlin_status launch_cache_dequant(const qlin_kv_cache& c, const int32_t* page_ids, int64_t n,
                                 void* out, cudaStream_t st);
size_t cache_attention_workspace_size(int head_dim);
qlin_status launch_cache_attention(const void* q, int64_t q_stride, void* out,
                                   const qlin_kv_cache& c, const int32_t* starts,
                                   int64_t n_tokens, int q_heads, float scale, int max_new,
                                   void* workspace, unsigned flags, cudaStream_t st);
// How a row of V logits, of M, is cut: CTAs that share it, elements of each one's
// part, and bits of the limbs that its weights are summed in.
struct SamplePlan {
  int ranks, part, limb;
};
SamplePlan sample_plan(int64_t M, int64_t V, int sms);
// a/tau as the kernel computes it, on the host.
float sample_quotient(float a, float tau);
qlin_status launch_sample(const void* logits, int64_t logits_stride, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p,
                          const float* min_p, int32_t* tokens, float* probs, int64_t M,
                          int64_t V, qlin_dtype ldtype, unsigned flags, cudaStream_t st);

qlin_status launch_token_logprobs(const void* logits, int64_t stride, const int32_t* tokens,
                                  float* logprobs, float* entropy, int top, int32_t* top_tokens,
                                  float* top_logprobs, int64_t M, int64_t V, qlin_dtype ldtype,
                                  unsigned flags, cudaStream_t st);

// ------------------------------------------------------------------ experts
// (route_experts.cu, expert_linear.cu, combine_experts.cu)
struct RouteArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  int scoring, groups, top_groups, group_score, top_k, renormalise;
  float scale;
  int32_t* experts;
  float* weights;
  int32_t* order;
  int32_t* offsets;
  int64_t T;
  int E;
  qlin_dtype dtype;
};
size_t route_experts_workspace_size(int64_t T, int E);
qlin_status launch_route_experts(const RouteArgs& r, void* workspace, unsigned flags,
                                 cudaStream_t st);

// Weights [E][N][K]; pair p's row of x is p / pairs_per_row.
struct ExpertArgs {
  const void* x;
  int64_t x_stride;
  int pairs_per_row;
  const int32_t* order;
  const int32_t* offsets;
  int64_t n_pairs;
  const uint32_t* wq;
  const void* scales;
  const void* biases;
  void* y;
  int y_f32;
  int E;
  int64_t N, K;
  void* workspace;
};
size_t expert_linear_workspace_size(int64_t n_pairs, int E, int64_t N, int64_t K);
qlin_status launch_expert_linear(const ExpertArgs& a, int bits, qlin_dtype dtype, unsigned flags,
                                 cudaStream_t st);
// The tensor-core kernel with a producer that stops before stage `stage` (for tests).
qlin_status launch_expert_stalled(const ExpertArgs& a, int stage, unsigned wait_limit_us,
                                  cudaStream_t st);
qlin_status launch_combine_experts(const void* y, const int32_t* experts, const float* weights,
                                   const void* add, int64_t add_stride, void* out, int64_t T,
                                   int top_k, int64_t N, qlin_dtype dtype, qlin_dtype y_dtype,
                                   unsigned flags, cudaStream_t st);

// Read and clear the kernels' device status words (no synchronisation).
cudaError_t qmm_take_device_status(unsigned* flags);
cudaError_t qmv_take_device_status(unsigned* flags);
cudaError_t chain_take_device_status(unsigned* flags);
cudaError_t rope_take_device_status(unsigned* flags);
cudaError_t attention_take_device_status(unsigned* flags);
cudaError_t sample_take_device_status(unsigned* flags);
cudaError_t expert_take_device_status(unsigned* flags);

constexpr int kGroup = 64;

}  // namespace qlin
