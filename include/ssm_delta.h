/*
 * ssm_delta.h -- C ABI of the gated delta rule on MI355X (gfx950): the chunked forward pass, the
 * single-token state update and the backward pass. Status codes, dtypes, ownership, streams and
 * error handling are those of ssm_scan.h.
 *
 * The operation, per batch entry and head, with a matrix state S of headdim x dstate (row p = one
 * channel of v; all arithmetic on the state fp32):
 *   S_t = a_t S_(t-1) + u_t k_t^T,   a_t = exp(g_t)
 *   u_t = beta_t (v_t - a_t S_(t-1) k_t)      the write corrects what the state holds for k_t
 *   y_t = scale S_t q_t
 * k plays the part of B, q of C, v of x of the selective scan with one decay per head; what is
 * new is the term S k in the write.
 *
 * Layouts. Element strides are given in the descriptor; the innermost dimension has stride 1:
 *   q, k        (batch, seqlen, ngroups, dstate)   io dtype; head h reads group
 *                                                   h / (nheads / ngroups)
 *   v, y        (batch, seqlen, nheads, headdim)   io dtype
 *   g, beta     (batch, seqlen, nheads)            io dtype; g is the logarithm of the decay
 *   states      (batch, nheads, headdim, dstate)   fp32 contiguous, the layout of the scan's
 *                                                   (batch, dim, dstate) states
 * Time is an outer dimension here (the scan's layout has it innermost): the rows of q, k and v are
 * the operands of the matrix products, and are what a projection writes.
 *
 * Steps are taken in chunks of 64 as matrix products: a NaN or an infinity in an input reaches,
 * beside the steps from its own on, the other steps of its chunk.
 *
 * Sizes that would take 2^32 threads in a launch (about 2^23 heads, or chunks of one group) return
 * SSM_ERR_UNSUPPORTED.
 */
#ifndef SSM_DELTA_H
#define SSM_DELTA_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_DELTA_MAX_DSTATE 128

/* Bits with which a value computed in fp32 (the state, a write, a weight within a chunk) enters a
 * matrix product of a call on bf16 tensors. All sums are fp32 in either case, and no output depends
 * on which other outputs are asked for. */
enum ssm_delta_operands {
  SSM_DELTA_OPERANDS_24 = 0, /* all of them: results as good as fp32 arithmetic makes them */
  SSM_DELTA_OPERANDS_16 = 1  /* 2^-17 of a value lost in each product; the states too are good to
                              * that. Faster (fp32 tensors: no difference). */
};

typedef struct ssm_delta_desc {
  int64_t batch;    /* >= 0 */
  int64_t seqlen;   /* L, >= 0 */
  int64_t nheads;   /* heads of v, g, beta and y, >= 1 */
  int64_t ngroups;  /* heads of q and k, >= 1, divides nheads */
  int64_t dstate;   /* entries of a key, 1..SSM_DELTA_MAX_DSTATE */
  int64_t headdim;  /* entries of a value, >= 1 */
  int32_t io_dtype; /* ssm_dtype of q, k, v, g, beta and y */
  int32_t operands; /* ssm_delta_operands; not used by ssm_gated_delta_update, which has no
                     * matrix products */
  int64_t q_stride_batch, q_stride_step, q_stride_group;
  int64_t k_stride_batch, k_stride_step, k_stride_group;
  int64_t v_stride_batch, v_stride_step, v_stride_head;
  int64_t g_stride_batch, g_stride_step, g_stride_head;
  int64_t beta_stride_batch, beta_stride_step, beta_stride_head;
  int64_t y_stride_batch, y_stride_step, y_stride_head;
} ssm_delta_desc;

/* Fills `desc` with the contiguous layout of the given sizes; sizes are checked by the calls that
 * use the descriptor. */
int ssm_delta_desc_init_contiguous(ssm_delta_desc* desc, int64_t batch, int64_t seqlen,
                                   int64_t nheads, int64_t ngroups, int64_t dstate,
                                   int64_t headdim, int32_t io_dtype);

/* Bytes of device workspace of ssm_gated_delta_fwd (depends only on the descriptor). There is room
 * in it for copies of q, k and v, made where their rows do not allow 16-byte access (also in the
 * backward pass's, and for dy). */
int ssm_gated_delta_workspace_size(const ssm_delta_desc* desc, size_t* bytes);

/* The forward pass.
 *   s0        : nullable initial state (zeros)
 *   s_final   : nullable; receives the state after the last step (s0, or zeros, when seqlen is 0)
 *   workspace : at least the queried size, 16-byte aligned
 * y, s_final and the workspace must not overlap any input or each other. */
int ssm_gated_delta_fwd(const ssm_delta_desc* desc, const void* q, const void* k, const void* v,
                        const void* g, const void* beta, float scale, const float* s0, void* y,
                        float* s_final, void* workspace, size_t workspace_bytes, void* stream);

/* One step per batch entry, for decoding: `desc` has seqlen 1 (SSM_ERR_BAD_SHAPE otherwise);
 * `state` is read and overwritten in place. state and y must not overlap any input or each other.
 * No workspace. */
int ssm_gated_delta_update(const ssm_delta_desc* desc, float* state, const void* q, const void* k,
                           const void* v, const void* g, const void* beta, float scale, void* y,
                           void* stream);

/* Bytes of device workspace of ssm_gated_delta_bwd (depends only on the descriptor). It holds the
 * state before and its gradient after every chunk of 64 steps. */
int ssm_gated_delta_bwd_workspace_size(const ssm_delta_desc* desc, size_t* bytes);

/* Gradients of ssm_gated_delta_fwd with respect to every input, given dy, the gradient of y (with
 * y's strides), and ds_final, that of the final state (nullable: zeros). The states are made again
 * from the inputs.
 *   dq, dk    : (batch, seqlen, ngroups, dstate) contiguous, io dtype, summed over the heads of a
 *               group
 *   dv        : (batch, seqlen, nheads, headdim) contiguous, io dtype
 *   dg, dbeta : (batch, seqlen, nheads) contiguous, io dtype
 *   ds0       : nullable; the gradient of the initial state (ds_final, or zeros, when seqlen is 0)
 *   workspace : at least the queried size, 16-byte aligned
 * Gradients are contiguous whatever the inputs' strides, so an input may be broadcast (stride 0).
 * Outputs must not overlap an input or each other. Sums are taken in a fixed order: results do not
 * vary from run to run. */
int ssm_gated_delta_bwd(const ssm_delta_desc* desc, const void* q, const void* k, const void* v,
                        const void* g, const void* beta, float scale, const float* s0,
                        const void* dy, const float* ds_final, void* dq, void* dk, void* dv,
                        void* dg, void* dbeta, float* ds0, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_DELTA_H */
