/*
 * zs_layers.h -- C ABI of the operators before, between and behind the products
 * of a block of experts, in the same library (libzs.so): lookup of rows by
 * token or species and its gradient, layer norm, routing to experts, and the
 * weighted sum of the experts' outputs.  The products themselves are
 * zs_grouped_mm (zs_block.h) over the CSR (zs.h) of the chosen experts.
 *
 * Conventions: those of zs_block.h (device pointers owned by the caller,
 * kernels on the current HIP device, asynchronous on `stream`, argument checks
 * on the host before any HIP call, negative zs_status codes, inputs never
 * written, outputs overlapping neither inputs nor each other; element types
 * per call; strides in elements with the last dimension contiguous; sums and
 * statistics in fp32 or more and each output rounded once; no allocation, no
 * synchronisation, no memset, so every call can be captured in a HIP graph;
 * no atomics, so results are the same bits from run to run).
 */
#ifndef ZS_LAYERS_H_
#define ZS_LAYERS_H_

#include "zs_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZS_MAX_LAYER_WIDTH 8192   /* channels of a row                        */
#define ZS_MAX_EXPERTS 1024       /* experts of a router                      */
#define ZS_MAX_SLOTS 64           /* experts that a row is sent to            */
#define ZS_MAX_EXPERT_GROUPS 64   /* groups of a router's experts             */

/*
 * zs_embedding -- y[i] = scale * table[index[i]], zeros where index[i] lies
 * outside [0, n_entries).
 *
 *   table    [n_entries][c], row stride table_stride       (input)
 *   index    [n_rows] int64                                (input)
 *   y        [n_rows][c] contiguous                        (output)
 */
int zs_embedding(const void *table, int64_t table_stride, const int64_t *index,
                 int64_t n_rows, int64_t n_entries, int64_t c, float scale,
                 int dtype, void *y, void *stream);

/*
 * zs_embedding_backward -- grad_table[v] = scale * sum of grad_y[i] over the
 * rows i with index[i] == v.  The sum is taken in fp32 in a fixed order that
 * depends on the sizes, offsets and perm alone: stretches of an entry's rows one
 * behind the other as perm has them, then the stretches' sums with one another.
 * It is not the sum of all rows one behind the other.
 *
 *   grad_y   [n_rows][c], row stride gy_stride             (input)
 *   index    [n_rows] int64, as in zs_embedding            (input)
 *   offsets  [n_entries + 1] int32, perm [n_rows] int32    (input)
 *            rowptr and perm of zs_build_csr over index (entries outside
 *            [0, n_entries) allowed, with a bad_flag), or perm NULL when the
 *            rows already are in the order of their entries: entry v's rows
 *            are offsets[v] .. offsets[v + 1] - 1.  Offsets and perm that do
 *            not belong to index give unspecified gradients but no access
 *            outside the arrays.
 *   grad_table [n_entries][c] contiguous, zeros for entries without a row
 *                                                          (output)
 *   workspace, workspace_bytes >= zs_embedding_backward_workspace_bytes(...),
 *            256-byte aligned device scratch (may be NULL when that is 0): the
 *            fp32 sums of entries whose rows are cut over workgroups
 */
size_t zs_embedding_backward_workspace_bytes(int64_t n_rows, int64_t c,
                                             int dtype);
int zs_embedding_backward(const void *grad_y, int64_t gy_stride,
                          const int64_t *index, const int32_t *offsets,
                          const int32_t *perm, int64_t n_rows,
                          int64_t n_entries, int64_t c, float scale, int dtype,
                          void *grad_table, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * zs_layer_norm -- y = (x - mu) (mean((x - mu)^2) + eps)^(-1/2) w + b, mu and
 * the mean over the c channels of a row.
 *
 *   x        [n_rows][c], row stride x_stride              (input)
 *   w, b     [c] fp32; b may be NULL (no bias)             (input)
 *   y        [n_rows][c] contiguous                        (output)
 * eps > 0.  Squares are summed in fp32: a row whose deviations from mu are
 * above some 1e19 / sqrt(c) has an infinite variance and gives b, and a sum of
 * x beyond fp32 gives NaN.  zs_layer_norm_backward recomputes the statistics from x; the
 * gradient of b is not written when grad_b is NULL.
 *   grad_y   [n_rows][c], row stride gy_stride             (input)
 *   grad_x   [n_rows][c] contiguous; grad_w, grad_b [c] fp32   (output)
 *   workspace: partial sums of grad_w and grad_b, added in a fixed order
 */
int zs_layer_norm(const void *x, int64_t x_stride, const float *w,
                  const float *b, int64_t n_rows, int64_t c, float eps,
                  int dtype, void *y, void *stream);
size_t zs_layer_norm_workspace_bytes(int64_t n_rows, int64_t c);
int zs_layer_norm_backward(const void *grad_y, int64_t gy_stride,
                           const void *x, int64_t x_stride, const float *w,
                           int64_t n_rows, int64_t c, float eps, int dtype,
                           void *grad_x, float *grad_w, float *grad_b,
                           void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * zs_route -- the experts of each row and their weights.
 *
 *   s = softmax(logits) or sigmoid(logits) of the row;  q = s + bias
 *   score of a group of n_experts / groups consecutive experts: the sum of its
 *     `best` largest q (one that has fewer: of those it has)
 *   the top_groups groups of largest score stay, and of their experts the k
 *     of largest q are chosen, in decreasing order
 *   weight = scale * s, or scale * s / sum of the chosen s (renormalise)
 *
 * An expert is there if its logit and its bias are above -inf (a NaN bias is
 * not).  Without bias the experts are ranked by their logits, which is the order
 * of s.  The choice is that of s, q and groups' scores in fp64, ties go to the
 * lowest index.  Weights are formed in fp64 and rounded once, but a softmax's
 * sum over all experts may be one of fp32 exponentials: without renormalise its
 * weights are off by up to 10 half ulps.  A row's results do not depend on the
 * other rows of a call.  A group without an expert does not stay.  A slot that
 * no expert is left for gets the index n_experts and weight 0.  Weights of a row
 * whose chosen scores are all 0 (sigmoid of logits below -709, renormalised) are
 * 0.  A row with a NaN logit, or in a softmax a logit of +inf, gets n_experts and
 * NaN in all slots.
 *
 *   logits   [n_rows][n_experts], row stride logits_stride (input)
 *   bias     [n_experts] fp32 or NULL                      (input)
 *   weight   [n_rows][k] fp32, expert [n_rows][k] int64    (output)
 *
 * The CSR of expert over n_experts + 1 nodes (zs_build_csr) groups the
 * n_rows * k slots for zs_grouped_mm; with its first n_experts + 1 row offsets
 * alone, slots without an expert are rows of no group.
 */
typedef struct zs_router {
    int32_t k;              /* 1 .. ZS_MAX_SLOTS, at most the experts that stay */
    int32_t sigmoid;        /* 0: softmax, 1: sigmoid                           */
    int32_t groups;         /* 1 .. ZS_MAX_EXPERT_GROUPS, divides n_experts     */
    int32_t top_groups;     /* 1 .. groups                                      */
    int32_t best;           /* 1 or 2                                           */
    int32_t renormalise;    /* 0 or 1                                           */
    float scale;
} zs_router;

int zs_route(const void *logits, int64_t logits_stride, const float *bias,
             const zs_router *router, int64_t n_rows, int64_t n_experts,
             int dtype, float *weight, int64_t *expert, void *stream);

/*
 * zs_route_backward -- gradient of the logits from that of the weights, the
 * choice held fixed (and no gradient for the bias, which only chooses).
 *
 *   grad_weight [n_rows][k] fp32, contiguous               (input)
 *   logits   as above; expert [n_rows][k] int64 from zs_route   (input)
 *   grad_logits [n_rows][n_experts] of logits' type, contiguous (output)
 * Slots whose index lies outside [0, n_experts) have no part in it, and a row
 * of such slots only gets zeros.  The chosen experts' gradients are formed in
 * fp64 and keep their digits where one of them has nearly all of a row; for a
 * sigmoid 1 - s is a difference of fp64 values, so above a logit of some 20 its
 * gradient is right to 2^-53 of grad_weight rather than of itself.
 */
int zs_route_backward(const float *grad_weight, const void *logits,
                      int64_t logits_stride, const int64_t *expert,
                      const zs_router *router, int64_t n_rows,
                      int64_t n_experts, int dtype, void *grad_logits,
                      void *stream);

/*
 * zs_combine -- y[t] = sum over j < k of weight[t][j] * z[t k + j].
 *
 *   z        [n_rows * k][c], row stride z_stride          (input)
 *   weight   [n_rows][k] fp32, contiguous                  (input)
 *   y        [n_rows][c] contiguous                        (output)
 * zs_combine_backward:
 *   grad_y   [n_rows][c], row stride gy_stride             (input)
 *   grad_z   [n_rows * k][c] contiguous: weight[t][j] * grad_y[t]   (output)
 *   grad_weight [n_rows][k] fp32: <grad_y[t], z[t k + j]>  (output)
 * 1 <= k <= ZS_MAX_SLOTS, n_rows * k at most ZS_MAX_EDGES.
 */
int zs_combine(const void *z, int64_t z_stride, const float *weight,
               int64_t n_rows, int64_t k, int64_t c, int dtype, void *y,
               void *stream);
int zs_combine_backward(const void *grad_y, int64_t gy_stride, const void *z,
                        int64_t z_stride, const float *weight, int64_t n_rows,
                        int64_t k, int64_t c, int dtype, void *grad_z,
                        float *grad_weight, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_LAYERS_H_ */
