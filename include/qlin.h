/*
 * qlin.h -- C ABI of libqlin: fused affine dequantise-into-matmul for
 * MLX-style packed 4/8-bit weights on NVIDIA GB300 (sm_103a).
 *
 * What the calls compute (the web pages the method comes from are cited by
 * title and section):
 *
 *   Packed weight format -- "epic: realize low-precision / quantized
 *   performance on the OpenXLA (IREE) backend", section Context: MLX 4/8-bit
 *   weights stay resident packed as a ui32 payload with one f16 (or, per
 *   "track(upstream-iree): fused dequant->matmul for the packed int8
 *   bandwidth win", section "What is already in-tree", bf16) scale and bias
 *   per group along K.
 *
 *   Reconstruction -- same section: bit-unpack, then w = q*scale + bias.
 *
 *   Fusion -- "track(upstream-iree): ...", section "The blocker (measured)":
 *   the matmul consumes the reconstructed weight; it is never written to DRAM.
 *
 *   M = 1 with N not a multiple of 4 -- "Metal backend: import qmv_impl from
 *   MLX": any N >= 1 is accepted.
 *
 * Shared notation and layouts (all row-major, all pointers are DEVICE
 * pointers owned by the caller; the library never allocates or frees):
 *
 *   bits        4 or 8; p = 32/bits codes per uint32 word
 *   group_size  64 (the only group size the kernels take; others return
 *               QLIN_ERR_UNSUPPORTED)
 *   W           N x K weights (output features x input features)
 *   wq          uint32 [N][K/p]; code k of row n sits at bits
 *               [bits*(k%p), bits*(k%p)+bits) of word wq[n][k/p]
 *               ("low bits first")
 *   scales,
 *   biases      sdtype [N][K/group_size]
 *   x           dtype [M][K]  (activations)
 *   y           dtype [M][N]  (y = x . W_hat^T, f32 accumulation, one
 *               round-to-nearest-even to dtype at the end)
 *
 * Errors: every call validates its arguments on the host before anything is
 * launched and returns a status; on failure nothing was launched and
 * qlin_last_error() (per calling thread) describes why.  The pages' own guards
 * likewise make unsupported settings fail fast instead of faulting mid-run
 * ("track(upstream-iree): ...", section "What is already in-tree").  A launch failure
 * reported by the CUDA runtime returns QLIN_ERR_CUDA.  Calls are asynchronous
 * on the given stream (a cudaStream_t passed as void*; NULL = legacy default
 * stream) and never synchronise the device.
 *
 * Device-side waits in the kernels are bounded; if one gives up it sets a
 * device status word that qlin_device_status() reads (and clears).
 */
#ifndef QLIN_H_
#define QLIN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QLIN_OK = 0,
  QLIN_ERR_INVALID_ARG = 1,  /* null pointer, non-positive size, K % group_size != 0, ... */
  QLIN_ERR_UNSUPPORTED = 2,  /* bits not in {4,8}, group_size != 64, dtype combination */
  QLIN_ERR_MISALIGNED = 3,   /* a pointer the 128-bit / TMA path needs 16-byte aligned is not */
  QLIN_ERR_CUDA = 4,         /* the CUDA runtime reported an error (see qlin_last_error) */
  QLIN_ERR_DEVICE_TIMEOUT = 5 /* a kernel's bounded wait gave up (qlin_device_status) */
} qlin_status;

typedef enum { QLIN_F32 = 0, QLIN_F16 = 1, QLIN_BF16 = 2 } qlin_dtype;

/* Human-readable name of a status code (static string).  No counterpart on
 * the pages: an addition of this library. */
const char* qlin_status_str(qlin_status s);

/* Detail of the last failing call made by this thread (static per-thread
 * buffer; empty string if none).  No counterpart on the pages: an addition of
 * this library, in the spirit of the guards that fail fast with a reason
 * ("track(upstream-iree): ...", section "What is already in-tree"). */
const char* qlin_last_error(void);

/* Library version as 10000*major + 100*minor + patch.  No counterpart on the
 * pages: an addition of this library. */
int qlin_version(void);

/*
 * Affine quantisation (load time; not on the per-token path).
 *   w       device float32 [N][K], finite values
 *   wq      device uint32 [N][K*bits/32]          (written)
 *   scales,
 *   biases  device sdtype [N][K/group_size]         (written)
 * Per row and group G of group_size consecutive k:
 *   scale = RNE_sdtype(fl32((max_G - min_G) / (2^bits - 1))),
 *   bias  = RNE_sdtype(min_G),
 *   q_k   = clamp(rint(fl32(fl32(w_k - bias) / scale)), 0, 2^bits - 1)
 *   (ties to even; q = 0 when the stored scale is 0).
 * The recipe is MLX's affine min/max quantisation with the rounding choices
 * spelled out (the pages give the format, not the quantiser).
 * sdtype: QLIN_F16 or QLIN_BF16.  Alignment: w and wq 16-byte aligned.
 */
qlin_status qlin_quantize_affine(const float* w, int64_t N, int64_t K, int bits, int group_size,
                                 qlin_dtype sdtype, uint32_t* wq, void* scales, void* biases,
                                 void* stream);

/*
 * Materialise the reconstruction w_hat[N][K] = RNE_out(q*scale + bias): one
 * correctly rounded step from the exact value, so it is bit-identical to a
 * host dequantisation (the pages require the in-graph reconstruction to match
 * the host dequant exactly: "track(upstream-iree): ...", section "What is
 * already in-tree").  out_dtype: QLIN_F32, or equal to
 * sdtype.  This is the unfused reference path and a test carrier; the matmul
 * entry points below never call it.  Alignment: wq and w_out 16-byte aligned.
 */
qlin_status qlin_dequant(const uint32_t* wq, const void* scales, const void* biases, int64_t N,
                         int64_t K, int bits, int group_size, qlin_dtype sdtype,
                         qlin_dtype out_dtype, void* w_out, void* stream);

/*
 * Fused matrix-vector / small-M product on CUDA cores (decode):
 *   y[m][n] = sum_k x[m][k] * (q[n][k]*scale[n][k/g] + bias[n][k/g])
 * for m < M, n < N.  dtype (QLIN_F16 or QLIN_BF16) is the type of x, y,
 * scales and biases.  Correct for any M >= 1 and N >= 1 (N need not be a
 * multiple of 4); fastest for M <= 4.  Alignment: x and wq 16-byte aligned.
 * Streams each packed word, scale and bias once per M-tile of 4 rows of x.
 * Defining passages: the reconstruction is consumed inside the product and
 * never written to DRAM ("track(upstream-iree): ...", section "The blocker
 * (measured)"); the M = 1 product for any N, including N not a multiple of 4
 * ("Metal backend: import qmv_impl from MLX").
 *
 * No workspace argument: the kernel gives each CTA whole rows and reduces
 * within a warp, so it needs no scratch memory, and the workspace pointer and
 * size query that a split-K design would need are not part of the call.
 */
qlin_status qlin_qmv(const void* x, const uint32_t* wq, const void* scales, const void* biases,
                     void* y, int64_t M, int64_t N, int64_t K, int bits, int group_size,
                     qlin_dtype dtype, void* stream);

/*
 * Launch flags for the *_ex entry points.  No counterpart on the pages: an
 * addition of this library, aimed at the launch gaps between dependent
 * linears (the pages count ~678 dispatches per packed decode step: "epic:
 * realize low-precision / quantized performance on the OpenXLA (IREE)
 * backend", section "The measured fusion gate").
 *
 * QLIN_OVERLAP_PREVIOUS: launch as a programmatic dependent launch.  The
 *   kernel may start while the preceding kernel on the stream is still
 *   running and begins streaming its weights, scales and biases at once; it
 *   reads x and writes y only after that kernel has completed and its writes
 *   are visible.  The caller guarantees that the preceding work on the stream
 *   does not write wq, scales or biases (true for resident weights in a
 *   decode loop).  Hides launch and ramp-up time between dependent launches.
 */
#define QLIN_OVERLAP_PREVIOUS 1u

/* qlin_qmv with launch flags (0 = same as qlin_qmv).  Unknown flag bits
 * return QLIN_ERR_INVALID_ARG.  Product as qlin_qmv (same passages); the
 * flags are an addition of this library. */
qlin_status qlin_qmv_ex(const void* x, const uint32_t* wq, const void* scales, const void* biases,
                        void* y, int64_t M, int64_t N, int64_t K, int bits, int group_size,
                        qlin_dtype dtype, unsigned flags, void* stream);

/*
 * A chain of dependent M = 1 products in one launch (a decode step).
 *
 * Link i computes y_i = x_i . W_hat_i^T with W_i given in the packed format
 * above (wq, scales, biases of shape [N][K]), where x_i is x0 (input = -1) or
 * the K elements starting at element input_offset of an earlier link's output
 * (0 <= input < i, input_offset + K <= N of that link).  The result is the
 * same as calling qlin_qmv on the links in order; the whole chain runs as one
 * persistent cooperative kernel whose CTAs stream every link's weights without
 * waiting and only wait, per link, until the row blocks of its input link are
 * complete.  The pages trace the packed path's slowness to unfused, separately
 * dispatched steps (~678 dispatches per decode step: "epic: realize
 * low-precision / quantized performance on the OpenXLA (IREE) backend",
 * section "The measured fusion gate").
 */
typedef struct {
  const uint32_t* wq;      /* [N][K*bits/32], 16-byte aligned */
  const void* scales;      /* dtype [N][K/group_size] */
  const void* biases;      /* dtype [N][K/group_size] */
  void* y;                 /* dtype [N] output; 16-byte aligned if a later link reads it */
  int64_t N, K;
  int32_t input;           /* -1: x0; else index of an earlier link */
  int32_t input_offset;    /* first element of that link's output read as x (x16 bytes aligned) */
} qlin_link;

/* Bytes of device scratch qlin_qmv_chain needs for n_links links (one 32-bit
 * completion counter per link, rounded up to 256 bytes).  No counterpart on
 * the pages: an addition of this library. */
size_t qlin_qmv_chain_workspace_size(int n_links);

/*
 * Run the chain.  x0: dtype [K of the links reading it], 16-byte aligned (may
 * be NULL when no link reads it).  workspace: device scratch of at least
 * qlin_qmv_chain_workspace_size(n_links) bytes, 16-byte aligned, owned by the
 * caller; the call zeroes it on the stream first, so concurrent chains need
 * separate workspaces.  1 <= n_links <= 160.  Outputs must not overlap any
 * weight or another link's output.  Errors as for qlin_qmv.
 */
qlin_status qlin_qmv_chain(const void* x0, const qlin_link* links, int n_links, int bits,
                           int group_size, qlin_dtype dtype, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * qlin_qmv_chain for callers that cannot allocate device memory (no
 * counterpart on the pages; an addition of this library).
 *
 * Same chain, same arguments and same results as qlin_qmv_chain, but the
 * per-link scratch counters live in a file-scope static device array inside
 * the library, so the call allocates nothing: for plugins whose host
 * framework owns all device memory through its own pool and forbids
 * cudaMalloc, and for deployments whose device memory budget is fixed at
 * start-up.  Limits: at most QLIN_CHAIN_STATIC_MAX_LINKS links (larger counts
 * return QLIN_ERR_INVALID_ARG); every GPU that loads the library keeps its
 * copy of the array until the process exits; all calls on a device share it
 * (each call zeroes the counters it uses on its stream first), so calls whose
 * kernels overlap on the GPU race and give wrong results.  The first call on
 * each device looks up the array's device address; make it before any stream
 * capture.
 */
#define QLIN_CHAIN_STATIC_MAX_LINKS 160
qlin_status qlin_qmv_chain_static(const void* x0, const qlin_link* links, int n_links, int bits,
                                  int group_size, qlin_dtype dtype, void* stream);

/*
 * The same product on the tensor cores (batched decode and prefill): packed
 * tiles are staged into shared memory by TMA, dequantised to dtype
 * (bit-identical to qlin_dequant's dtype output) into tensor memory as the
 * A operand of tcgen05 MMAs with f32 accumulators in tensor memory; when the
 * output has few tiles, K is split over a thread-block cluster and the
 * partial sums are added through distributed shared memory (no workspace).
 * Same arguments and result contract as qlin_qmv: for dtype QLIN_BF16 the
 * tensor-core operand carries w_hat as bf16 hi plus a bf16 residual lo (two
 * MMAs per K step), so rounding the operand to bf16 costs no accuracy.  Extra
 * requirement: K % 64 == 0 (always true for group 64) and x, wq 16-byte
 * aligned.  Defining passages: the target must fuse the dequantisation into
 * the matmul ("track(upstream-iree): ...", sections "The blocker (measured)"
 * and "Unblock criteria"), with bf16 scales and biases accepted (same page,
 * "What is already in-tree").
 */
qlin_status qlin_qmm(const void* x, const uint32_t* wq, const void* scales, const void* biases,
                     void* y, int64_t M, int64_t N, int64_t K, int bits, int group_size,
                     qlin_dtype dtype, void* stream);

/* qlin_qmm with launch flags (0 = same as qlin_qmm).  QLIN_OVERLAP_PREVIOUS
 * as for qlin_qmv_ex: the launch and the kernel's set-up (barriers, tensor
 * memory, descriptor prefetch) overlap the preceding kernel on the stream; x
 * is read and y written only after that kernel has completed.  Unknown flag
 * bits return QLIN_ERR_INVALID_ARG.  Product as qlin_qmm (same passages); the
 * flags are an addition of this library. */
qlin_status qlin_qmm_ex(const void* x, const uint32_t* wq, const void* scales, const void* biases,
                        void* y, int64_t M, int64_t N, int64_t K, int bits, int group_size,
                        qlin_dtype dtype, unsigned flags, void* stream);

/*
 * Dispatch to qlin_qmv when M < qlin_crossover_m_dtype(N, K, bits, dtype), else
 * qlin_qmm.
 * The product is the one both kernels define (same passages); choosing
 * between them by M is an addition of this library.
 */
qlin_status qlin_linear(const void* x, const uint32_t* wq, const void* scales,
                        const void* biases, void* y, int64_t M, int64_t N, int64_t K, int bits,
                        int group_size, qlin_dtype dtype, void* stream);

/* Smallest M for which qlin_linear picks the tensor-core path for activation
 * dtype `dtype`, from measurements on GB300: 4 for f16 when K > N; else 5
 * when N*K >= 6*2^20 and 9 below (qmv reads the weights once per 4 tokens).
 * `bits` does not change it (4- and 8-bit measured alike).  The environment
 * variable QLIN_CROSSOVER_M (read once per process) overrides it.  No
 * counterpart on the pages: an addition of this library. */
int64_t qlin_crossover_m_dtype(int64_t N, int64_t K, int bits, qlin_dtype dtype);

/* qlin_crossover_m_dtype for f16 activations. */
int64_t qlin_crossover_m(int64_t N, int64_t K, int bits);

/*
 * qlin_linear with a linear layer's epilogue:
 *
 *   y[m][n] = RNE_ydtype( sum_k x[m][k] * w_hat[n][k]  +  layer_bias[n] )
 *
 * layer_bias: dtype [N] (the activation dtype), added to the f32 accumulator
 *   before the single final rounding; NULL for no bias.  (This is the layer's
 *   own bias vector, not the quantisation biases of the packed format.)
 * y_dtype: QLIN_F32 (y is float [M][N], 4-byte aligned, no rounding) or the
 *   activation dtype (y as in qlin_linear).
 * The pages' ExecuTorch stack ships a 4-bit linear with bias ("Metal backend:
 * import qmv_impl from MLX", its stack of changes: "enable linear with bias",
 * "test 4-bit linear with bias"); the f32 output serves callers that keep the
 * residual stream in f32 (an addition of this library).
 *
 * Errors: as qlin_linear; y_dtype other than QLIN_F32 or dtype is
 * QLIN_ERR_UNSUPPORTED; layer_bias not 2-byte or an f32 y not 4-byte aligned
 * is QLIN_ERR_MISALIGNED.
 */
qlin_status qlin_linear_ex(const void* x, const uint32_t* wq, const void* scales,
                           const void* biases, const void* layer_bias, void* y, int64_t M,
                           int64_t N, int64_t K, int bits, int group_size, qlin_dtype dtype,
                           qlin_dtype y_dtype, void* stream);

/* ==========================================================================
 * What stands between a decoder's linears: RMS norm with the residual's
 * addition, rotary positions with the append to an 8-bit key/value cache,
 * attention over that cache, and sampling.  None has a counterpart on the
 * pages, whose decode step is its linears; these are additions of this library.
 *
 * flags of the calls below: 0 or QLIN_OVERLAP_PREVIOUS (the launch and what
 * reads no tensor of the call overlap the preceding kernel on the stream).
 *
 * Head dimensions 64 and 128; activations f16 or bf16.
 * ======================================================================== */

/*
 * The key/value cache of one layer.  A slot is one sequence.  Tokens are kept
 * in blocks of QLIN_KV_BLOCK: complete blocks in 8 bits, in pages that the
 * table names in any order, with one float32 scale for each block, head and
 * key/value; the incomplete last block (the slot's tail) in dtype.  Every
 * value is therefore rounded to 8 bits once, when its block completes, and
 * what the cache holds does not depend on how the tokens were grouped in
 * calls.  A code c stands for (c - 128) * scale, 1 <= c <= 255.  Value blocks
 * are held transposed, as the attention's products read them.  Pages may be
 * shared by slots with a common beginning.
 *
 *   pages    uint8 [n_pages][kv_heads][2][64*head_dim]: keys as
 *            [64 tokens][head_dim], then values as [head_dim][64 tokens]
 *   scales   float [n_pages][kv_heads][2]
 *   tail     dtype [slots][kv_heads][2][64*head_dim], same two layouts;
 *            what stands beyond a slot's last token is never used
 *   table    int32 [slots][max_blocks]: the page of each block
 *   lens     int32 [slots]: tokens held before the call (shared by a model's
 *            layers; the caller advances it once per step)
 *
 * At most 1024 slots.  pages and tail are 16-byte aligned.  The struct is read
 * during the call only; the memory it names is used on the stream.
 */
#define QLIN_KV_BLOCK 64
typedef struct {
  void* pages;
  float* scales;
  void* tail;
  const int32_t* table;
  const int32_t* lens;
  int64_t n_pages;
  int32_t slots, max_blocks, kv_heads, head_dim;
  int32_t dtype; /* a qlin_dtype: QLIN_F16 or QLIN_BF16 */
} qlin_kv_cache;

/*
 * y[m][k] = h * weight[k] / sqrt(mean_k(h*h) + eps),  h = x[m][k] + residual[m][k]
 *
 * x, weight and y are dtype; residual and residual_out are rdtype (dtype or
 * QLIN_F32).  h is a float32 sum: the norm uses it unrounded, residual_out
 * receives it rounded once to rdtype.  residual may be NULL (h = x), and then
 * residual_out is NULL too; residual_out may be NULL.  residual_out may be
 * residual, and y may be x, for use in place.  x_stride and residual_stride
 * are elements from row to row (>= K); y and residual_out are contiguous, so
 * use in place wants the same.  1 <= K <= 32768.  Alignment: of the elements
 * (rows that start 16-byte aligned are the fast path).
 */
qlin_status qlin_add_rms_norm(const void* x, int64_t x_stride, const void* weight,
                              const void* residual, int64_t residual_stride, void* residual_out,
                              void* y, int64_t M, int64_t K, float eps, qlin_dtype dtype,
                              qlin_dtype rdtype, unsigned flags, void* stream);

/*
 * Load time: the table of rotary positions, float [n_positions][rot_dim/2][2],
 * (cos, sin) of position * f_i, f_i = base^(-2i/rot_dim), computed in 64 bits.
 * Long contexts: factor > 1 divides the frequencies whose wavelength
 * 2*pi/f_i is above long_wavelength (0: all of them, plain interpolation) by
 * factor, leaves those below short_wavelength as they are, and blends between
 * the two, linearly in 1/wavelength.  factor = 1 scales nothing.
 * INVALID_ARG: rot_dim not a positive multiple of 2, base <= 1, factor < 1,
 * negative wavelengths or short_wavelength > long_wavelength.
 */
qlin_status qlin_rope_table(float* table, int64_t n_positions, int rot_dim, double base,
                            double factor, double short_wavelength, double long_wavelength,
                            void* stream);

/*
 * Rotates the queries and keys of new tokens and appends keys and values to
 * the cache.
 *   qkv      dtype [n_tokens][qkv_stride]: a row holds q_heads queries, then
 *            kv_heads keys, then kv_heads values of head_dim
 *   q_out    dtype [n_tokens][q_heads][head_dim]
 *   table    float [n_positions][rot_dim/2][2] (qlin_rope_table)
 *   starts   int32 [slots+1]: slot b's new tokens are rows starts[b] ..
 *            starts[b+1]-1, in order, at positions lens[b], lens[b]+1, ...
 *            (no rows: the slot is left as it is)
 * The first rot_dim elements of a head turn in pairs, the rest stays:
 * interleaved = 0 pairs i with i + rot_dim/2, 1 pairs 2i with 2i + 1;
 * (a, b) -> (a cos - b sin, b cos + a sin) in float32, rounded once to dtype.
 * Values and rotated keys enter the cache as dtype; a block that the call
 * completes gets scale = amax/127 and codes rint(v/scale) + 128 (float32,
 * ties to even; 128 where the scale is 0).  A block with an element that is
 * not finite (in dtype: the rotation can pass f16's range) gets the scale
 * infinity and codes 128: it stands for NaN.
 * rot_dim: a multiple of 16, 0 .. head_dim.  qkv and q_out 16-byte aligned
 * and apart, qkv_stride a multiple of 8.  A slot whose blocks pass max_blocks, a page
 * outside n_pages, a position outside the table or rows outside n_tokens are
 * left out and set a device status bit (qlin_device_status).
 */
qlin_status qlin_rope_append(const void* qkv, int64_t qkv_stride, void* q_out,
                             const float* table, int64_t n_positions, int rot_dim,
                             int interleaved, const qlin_kv_cache* cache, const int32_t* starts,
                             int64_t n_tokens, int q_heads, unsigned flags, void* stream);

/* The values that n pages of the cache stand for, out dtype
 * [n][kv_heads][2][64*head_dim] in the pages' layouts (16-byte aligned):
 * (c - 128) * scale in float32, rounded once.  page_ids: int32 [n] on the
 * device; a page outside n_pages gives zeros and sets a device status bit. */
qlin_status qlin_cache_dequant(const qlin_kv_cache* cache, const int32_t* page_ids, int64_t n,
                               void* out, void* stream);

/* Bytes of scratch that qlin_cache_attention needs for this head dimension on
 * the current device (0 for a head dimension it does not take). */
size_t qlin_cache_attention_workspace_size(int head_dim);

/*
 * Attention of new tokens over the cache that already holds them
 * (qlin_rope_append before, with the same lens and starts):
 *   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale * q[t][h] . k_j)
 * over the positions j <= lens[b] + i of slot b, whose i-th row is t; query
 * head h reads key/value head h / (q_heads/kv_heads).
 *   q        dtype [n_tokens][q_stride], heads contiguous in a row
 *   out      dtype [n_tokens][q_heads][head_dim]
 *   max_new  the most new tokens of any slot (host side; it chooses kernels
 *            and may be larger than it needs to be; a slot with more is left
 *            out, zeros in its rows, and sets a device status bit)
 *   workspace  qlin_cache_attention_workspace_size(head_dim) bytes of device
 *            memory, 16-byte aligned, with anything in it; calls that can
 *            overlap need workspaces of their own
 * What a row does not see does not reach it, whether it is finite or not; a
 * value that it sees and that is not finite makes it so.
 * Scores, softmax statistics and sums are float32; exponentials are the
 * hardware's (2 ulp).  Rounded to 16 bits on the way: probabilities, to f16 in
 * units of the largest product of a probability and its block's value scale so
 * far (2^-11 of each, or 2^-25 of that unit; a bf16 tail of few rows keeps 16
 * bits of them); bf16 queries, to f16 after a power of two for each row (exact
 * down to 2^-28 of the row's largest); with many rows a bf16 tail in the same
 * way.  f16 outputs are up to 30% further from the exact ones than by their own
 * rounding alone, bf16 ones 1%.
 * q_heads: a multiple of kv_heads, at most 16 times as many.  q and out 16-byte
 * aligned and apart, q_stride a multiple of 8.  Rows that no slot owns are not
 * written; blocks whose page is outside n_pages are left out and set a device
 * status bit.
 */
qlin_status qlin_cache_attention(const void* q, int64_t q_stride, void* out,
                                 const qlin_kv_cache* cache, const int32_t* starts,
                                 int64_t n_tokens, int q_heads, float scale, int max_new,
                                 void* workspace, size_t workspace_bytes, unsigned flags,
                                 void* stream);

/*
 * One token per row of logits, ldtype [M][V] (QLIN_F32, F16 or BF16; rows
 * logits_stride elements apart), from a given uniform number u[m] in [0, 1).
 * All parameters are device arrays of M values.
 *   w_i = rint(2^36 * exp((x_i - max)/temperature)): whole numbers, so sums
 *         are exact and a draw does not depend on how the work is split
 *   order: larger logits first, equal ones by index
 *   top_k       keeps the first k (<= 0: all)
 *   top_p       keeps, of those, each whose predecessors hold less than top_p
 *               of their mass (>= 1: all)
 *   min_p       keeps what is at least min_p times as likely as the likeliest
 *   The first of the order is always kept.  The token is the first index, in
 *   index order, whose cumulated kept weight is above floor(u * total);
 *   probs[m] is its share of the kept weight.
 * temperature <= 0: the first of the order, probability 1.  NaN logits count
 * as -infinity; a row of nothing else gives token -1, probability 0; with
 * +infinity among the logits only those can be drawn.  u outside [0, 1) is
 * taken into it.  1 <= V <= 262144.  probs may be NULL.
 */
qlin_status qlin_sample(const void* logits, int64_t logits_stride, const float* u,
                        const float* temperature, const int32_t* top_k, const float* top_p,
                        const float* min_p, int32_t* tokens, float* probs, int64_t M, int64_t V,
                        qlin_dtype ldtype, unsigned flags, void* stream);

/*
 * Read and clear the device status words of the current device (synchronises
 * the device).  *flags receives 0 when no kernel gave up a bounded wait since
 * the last call, else a bit mask of the waits that gave up (bits 0-7: the
 * tensor-core kernel, bits 8-15: the CUDA-core kernel, bits 16-23: the chain
 * kernel), or of what the cache kernels refused on the device (bit 24: rows
 * outside n_tokens or a negative length, 25: a page outside n_pages or a slot
 * past max_blocks, 26: a position outside the table, 27: a slot with more than
 * max_new rows, 28: a wait of the attention kernel that gave up), or in sampling
 * (bit 29: a bound that no bin passed was left out).  Returns QLIN_OK, or
 * QLIN_ERR_CUDA if the device could not be read.  No counterpart on the pages:
 * an addition of this library (a kernel that gives up a wait reports instead
 * of hanging, the device-side form of failing fast).
 */
qlin_status qlin_device_status(int* flags);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_H_ */
