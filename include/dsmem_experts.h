/*
 * dsmem_experts -- an expert layer's operators for NVIDIA GB300 (sm_103a):
 * routing, grouping by key, products grouped by key, the weighted way back,
 * and the gradients' global norm with clipping.
 *
 * dsmem_hist counts how many keys each owner has.  These calls go on from
 * there: they put rows in the order of their keys (dsmem_group), multiply
 * each group's rows with the group's own matrix (dsmem_grouped_matmul, and
 * its two gradients), bring the rows back to the tokens they came from
 * (dsmem_combine), choose the keys from a router's scores (dsmem_route), and
 * clip the gradients that come out (dsmem_grad_clip).
 *
 * Conventions are those of dsmem_hist.h: 0 or a negative DSMEM_HIST_E* code,
 * dsmem_hist_last_error() for the message, device pointers on the current
 * device, work enqueued on `stream` without synchronising, scratch (where a
 * call says it takes some) from the library's stream-ordered pool, and bad
 * arguments refused before anything is enqueued.  Outputs are overwritten.
 * Device contents are never trusted for addressing: keys, ids, offsets,
 * orders and positions that are out of range read and write nothing outside
 * the stated buffers.
 *
 * The calls can be captured into a CUDA graph once one has run on the device.
 * Such a graph reports to the captured stream's status word, so it is not
 * replayed after dsmem_hist_release().
 *
 * The same call gives the same bits: sums are taken in an order that sizes and
 * the device alone decide, in 32 bits or more, and rounded once to the output's
 * type.
 *
 * The product kernels wait for their own copies and matrix instructions with
 * bounded waits (about 50 ms each).  A wait that gives up makes the launch's
 * output wrong and is reported as in dsmem_hist.h: the next call on the same
 * stream returns DSMEM_HIST_ETIMEOUT and enqueues nothing, and
 * dsmem_hist_device_status() shows bit 1 (after the last product of a step, which
 * no call follows, ask there once the stream has been synchronised).  The test hooks of dsmem_hist.h hold
 * here too: DSMEM_HIST_TEST_WAIT_CYCLES bounds these waits,
 * DSMEM_HIST_TEST_WITHHOLD_LAST_ROUND leaves out the copies of the last stage of
 * depth, so that the wait for them runs out with none of them in flight, and
 * DSMEM_HIST_TEST_FAIL_ALLOC fails the calls that take scratch.
 */
#ifndef DSMEM_EXPERTS_H
#define DSMEM_EXPERTS_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#include "dsmem_hist.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { DSMEM_F32 = 0, DSMEM_F16 = 1, DSMEM_BF16 = 2 };

#define DSMEM_ROUTE_MAX_EXPERTS 1024
#define DSMEM_ROUTE_MAX_TOP_K 32
#define DSMEM_GROUP_MAX_GROUPS 32768
#define DSMEM_PRODUCT_MAX_GROUPS 2048

/* Chooses each token's experts.  Per row of `logits` [tokens, experts]:
 * ids[t, j] is the expert of the j-th largest logit, equal logits going to
 * the lowest index, and weights[t, j] its share of the softmax over the row,
 * or (renormalize != 0) over the chosen ones.  A logit of -inf or NaN is
 * masked: it is never chosen and has no share.  Where fewer than top_k are
 * left (none, in a masked row) the remaining ids are -1 and their weights 0.
 * Logits of +inf share the whole weight equally.
 *   dtype       of the logits: DSMEM_F32, DSMEM_F16 or DSMEM_BF16
 *   row_stride  elements between rows (>= experts)
 *   experts     1 .. 1024;  top_k 1 .. min(experts, 32)
 *   ids         int32 [tokens, top_k];  weights float [tokens, top_k] */
DSMEM_HIST_API int dsmem_route(const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                               int64_t row_stride, int32_t top_k, int32_t renormalize, int32_t* ids,
                               float* weights, cudaStream_t stream);

/* Gradient of dsmem_route's weights with respect to the logits; `ids` and
 * `weights` are the forward call's.  grad_logits [tokens, experts] has the
 * logits' type and is contiguous; masked logits get 0. */
DSMEM_HIST_API int dsmem_route_backward(const void* logits, int32_t dtype, int64_t tokens,
                                        int32_t experts, int64_t row_stride, int32_t top_k,
                                        int32_t renormalize, const int32_t* ids,
                                        const float* weights, const float* grad_weights,
                                        void* grad_logits, cudaStream_t stream);

/* Stable grouping of n keys (0 <= n < 2^31): with c(g) the histogram of the
 * keys in [0, num_groups) and others dropped,
 *   offsets[g]   = c(0) + .. + c(g-1),            g = 0 .. num_groups
 *   position[i]  = offsets[keys[i]] + number of i' < i with the same key; -1 if dropped
 *   order[p]     = the i with position[i] == p;   -1 for p >= offsets[num_groups]
 *   num_groups  1 .. 32768
 *   offsets int32 [num_groups + 1], order and position int32 [n]
 * Takes scratch from the pool for more than 2^18 keys, and for more than 12,288
 * into 17,057 groups or more. */
DSMEM_HIST_API int dsmem_group(const int32_t* keys, int64_t n, int32_t num_groups, int32_t* offsets,
                               int32_t* order, int32_t* position, cudaStream_t stream);

/* Products grouped by key.  Row p of the output belongs to group g where
 * offsets[g] <= p < offsets[g+1] (offsets[0] counts as 0), and its source row
 * is order[p] / fan, or p when `order` is NULL:
 *   transpose == 0:  out[p, :] = x[row(p), :] weight[g]^T   x [x_rows, inner], out [n, outer]
 *   transpose != 0:  out[p, :] = x[row(p), :] weight[g]     x [x_rows, outer], out [n, inner]
 * with weight [groups, outer, inner].  Rows p of no group, and rows whose
 * source lies outside x, are 0.
 *   dtype       of x and weight: DSMEM_F16 or DSMEM_BF16; products are summed
 *               in 32 bits
 *   out_dtype   `dtype` or DSMEM_F32
 *   *_stride    elements between rows, at least a row's length, and
 *               weight_group_stride between groups, at least 1: views that repeat
 *               a row or a matrix by a stride of 0 are refused.  Rows themselves
 *               are contiguous, and out's rows too
 *   groups      1 .. 2048;  x_rows, n, outer, inner < 2^31 - 512
 * All such sizes and strides, and any alignment of the elements, are right.
 * Sources whose base, row
 * stride and group stride are multiples of 16 bytes are read in place; others
 * are first laid out so in pool scratch (one more pass over them). */
DSMEM_HIST_API int dsmem_grouped_matmul(const void* x, int64_t x_rows, int64_t x_stride,
                                        const void* weight, int64_t weight_row_stride,
                                        int64_t weight_group_stride, const int32_t* offsets,
                                        int32_t groups, const int32_t* order, int32_t fan, int64_t n,
                                        int32_t outer, int32_t inner, int32_t transpose,
                                        int32_t dtype, void* out, int32_t out_dtype,
                                        cudaStream_t stream);

/* Gradient of dsmem_grouped_matmul (transpose == 0) with respect to the
 * weights:  out[g] = sum over p of group g of dy[p, :]^T x[row(p), :], and 0
 * for an empty group.  dy [n, outer], x [x_rows, inner], out [groups, outer,
 * inner], contiguous.  Arguments as there. */
DSMEM_HIST_API int dsmem_grouped_matmul_wgrad(const void* dy, int64_t dy_stride, const void* x,
                                              int64_t x_rows, int64_t x_stride,
                                              const int32_t* offsets, int32_t groups,
                                              const int32_t* order, int32_t fan, int64_t n,
                                              int32_t outer, int32_t inner, int32_t dtype, void* out,
                                              int32_t out_dtype, cudaStream_t stream);

/* Brings grouped rows back:  out[t, :] = sum over j, in order, of
 * weights[t, j] * z[position[t, j], :] over the positions in [0, z_rows);
 * others (dropped) are not read, and a token without any is 0.
 *   weights  float [tokens, top_k], or NULL for 1
 *   dtype    of z and out: DSMEM_F32, DSMEM_F16 or DSMEM_BF16
 *   z        [z_rows, width], z_stride >= width elements between rows; out
 *            contiguous
 *   width    1 .. 2^31 - 2049;  tokens * top_k < 2^31 */
DSMEM_HIST_API int dsmem_combine(const void* z, int64_t z_rows, int64_t z_stride,
                                 const int32_t* position, const float* weights, int64_t tokens,
                                 int32_t top_k, int32_t width, int32_t dtype, void* out,
                                 cudaStream_t stream);

/* Gradients of dsmem_combine:  dz[position[t, j], :] = weights[t, j] * dy[t, :]
 * and dweights[t, j] = <dy[t, :], z[position[t, j], :]> (0 where dropped).
 * `position` and `order` are one dsmem_group call's, with tokens * top_k
 * keys; rows p of dz with order[p] < 0 are 0.
 *   dy       [tokens, width], dy_stride >= width elements between rows
 *   z        [tokens * top_k, width], z_stride >= width elements between rows
 *   weights  not NULL (ones for a combination without)
 *   dz       [tokens * top_k, width] contiguous;  dweights float [tokens, top_k] */
DSMEM_HIST_API int dsmem_combine_backward(const void* dy, int64_t dy_stride, const void* z,
                                          int64_t z_stride, const int32_t* position,
                                          const int32_t* order, const float* weights, int64_t tokens,
                                          int32_t top_k, int32_t width, int32_t dtype, void* dz,
                                          float* dweights, cudaStream_t stream);

/* One gradient of dsmem_grad_clip. */
typedef struct dsmem_grad {
  const void* grad; /* device, `count` elements, contiguous */
  void* out;        /* device, `count` elements of the same type; may be `grad` itself */
  int64_t count;    /* >= 0 */
  int32_t dtype;    /* DSMEM_F32, DSMEM_F16 or DSMEM_BF16 */
  int32_t reserved; /* 0 */
} dsmem_grad_t;

/* Global norm and clipping:  *norm = sqrt(sum of all squares), and every
 * out = grad * min(1, max_norm / (*norm + 1e-6)).  A norm that is infinite or
 * NaN goes through the formula.  No gradient overlaps another, nor another's out.
 *   grads     HOST array of num_grads entries (read before the call returns)
 *   max_norm  positive and finite (FLT_MAX for the norm alone)
 *   norm      device, one float
 * Takes scratch from the pool. */
DSMEM_HIST_API int dsmem_grad_clip(const dsmem_grad_t* grads, int32_t num_grads, float max_norm,
                                   float* norm, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSMEM_EXPERTS_H */
