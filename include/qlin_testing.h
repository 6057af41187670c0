/*
 * qlin_testing.h -- entry points of libqlin that exist only for the library's
 * own tests: to reach failure paths without faulting or hanging a GPU, and to
 * check host-side launch choices without one.  They have no counterpart on
 * the pages the method comes from, and no product code calls them.
 */
#ifndef QLIN_TESTING_H_
#define QLIN_TESTING_H_

#include "qlin.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * qlin_qmv_chain with one dependency that can never be met: the links that
 * read link `stalled_link` wait for one more completed row block than that
 * link has, so their bounded wait runs out after `wait_limit_us`
 * microseconds (1 .. 2,000,000).  The kernel then records bit 2 of the chain
 * kernel's status (qlin_device_status reports 1 << 18), carries on with
 * whatever the input holds (those outputs are garbage), lets every bulk copy
 * it issued land, and exits; the context stays usable.  Arguments otherwise
 * as qlin_qmv_chain.  Errors: QLIN_ERR_INVALID_ARG when stalled_link is out of
 * range or no later link reads it, or wait_limit_us is out of range; else as
 * qlin_qmv_chain.
 */
qlin_status qlin_testing_qmv_chain_stalled(const void* x0, const qlin_link* links, int n_links,
                                           int bits, int group_size, qlin_dtype dtype,
                                           void* workspace, size_t workspace_bytes,
                                           int stalled_link, unsigned wait_limit_us,
                                           void* stream);

/*
 * qlin_expert_linear (4 bits, QLIN_F16) by the tensor-core kernel, where in each CTA the
 * copies of packed weights stop before its stage `stalled_stage` (a group of 64 of K of
 * a tile; the CTA's tiles one after another): every wait behind them runs out after
 * `wait_limit_us` microseconds (1000 .. 2,000,000).  The kernel then records its status
 * (qlin_device_status reports 1 << 30), lets its copies and products in flight end,
 * frees its tensor memory and exits; outputs of tiles that were not complete are not
 * written, and the context stays usable.  A CTA with no more stages than that runs as
 * ever.  Arguments otherwise as qlin_expert_linear.  Errors: QLIN_ERR_INVALID_ARG where
 * the call needs no workspace (it would not take that kernel), stalled_stage is negative
 * or wait_limit_us out of range; else as qlin_expert_linear.
 */
qlin_status qlin_testing_expert_linear_stalled(
    const void* x, int64_t x_stride, int pairs_per_row, const int32_t* order,
    const int32_t* offsets, int64_t n_pairs, const uint32_t* wq, const void* scales,
    const void* biases, void* y, int E, int64_t N, int64_t K, void* workspace,
    size_t workspace_bytes, int stalled_stage, unsigned wait_limit_us, void* stream);

/*
 * The split of K that qlin_qmv (and qlin_linear's qmv path) would use for an
 * N x K matrix of `bits`-bit codes on a device with `sm_count` SMs: the
 * number of CTAs (a thread-block cluster) that share each row block, each
 * taking an equal share of the row's k-tiles (1: no split).  Host logic only;
 * touches no device.  Honours the QLIN_QMV_SPLIT and QLIN_QMV_R tuning
 * variables as the launcher does.  Returns -1 for arguments qlin_qmv would
 * reject (bits not 4 or 8, K not a positive multiple of 64, N < 1) or
 * sm_count < 1.
 */
int qlin_testing_qmv_split(int64_t N, int64_t K, int bits, int sm_count);

/*
 * How qlin_sample cuts each of M rows of V logits on a device with `sm_count`
 * SMs: *ranks CTAs (a thread-block cluster) share a row, each takes *part
 * consecutive elements (the last ones what is left of them), and all sum
 * weights in limbs of *limb_bits bits.  Host logic only; touches no device.
 * Returns QLIN_ERR_INVALID_ARG for M < 1, V outside 1 .. 262144, sm_count < 1
 * or a null pointer.
 */
qlin_status qlin_testing_sample_plan(int64_t M, int64_t V, int sm_count, int* ranks, int* part,
                                     int* limb_bits);

/*
 * q[i] = a[i]/tau[i] by the steps that qlin_sample takes in place of a division
 * (same fused multiply-adds, on the host; a, tau and q are HOST pointers), for
 * i < n.  Returns QLIN_ERR_INVALID_ARG for n < 0 or a null pointer.
 */
qlin_status qlin_testing_sample_quotient(const float* a, const float* tau, float* q, int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_TESTING_H_ */
