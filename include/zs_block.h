/*
 * zs_block.h -- C ABI of the learned operators around the zonal scatter, in the
 * same library (libzs.so): matrix products grouped by species or expert, the
 * gated residual join between two norms, and the AdamW step over all of a
 * model's parameter tensors.
 *
 * Conventions: those of zs.h (device pointers owned by the caller, kernels on
 * the current HIP device, asynchronous on `stream`, argument checks on the
 * host before any HIP call, negative zs_status codes, inputs never written,
 * outputs overlapping neither inputs nor each other).  In addition:
 *  - Element types are given per call (zs_dtype).  Sums and statistics are
 *    fp32 whatever the type; each output is rounded to its type once.
 *  - Strides are in elements, the last dimension is contiguous, and a view
 *    spans at most 2^60 elements.
 *  - No call allocates, synchronises or records a memset, so all of them can
 *    be captured in a HIP graph.  A captured AdamW step is not the next step
 *    at each replay but its own again (see zs_adamw_step).
 *  - Results are run-to-run deterministic (no atomics).
 */
#ifndef ZS_BLOCK_H_
#define ZS_BLOCK_H_

#include "zs.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum zs_dtype {
    ZS_F32 = 0,
    ZS_BF16 = 1
} zs_dtype;

#define ZS_MAX_GROUPS 1048576    /* groups of a grouped product               */
#define ZS_MAX_WIDTH 65536       /* k and n of a grouped product              */
#define ZS_MAX_JOIN_WIDTH 8192   /* channels of a residual join               */
#define ZS_ADAMW_BLOCK 256       /* elements that share a scale (8-bit state) */

/*
 * zs_grouped_mm -- y[i] = x[i] op(w[g(i)]), rows grouped by species or expert.
 *
 *   x        [n_rows][k], row stride x_stride             (input)
 *   w        [n_groups][k][n] (w_transposed == 0) or [n_groups][n][k]
 *            (w_transposed != 0), group stride w_group_stride, row stride
 *            w_stride                                     (input)
 *   offsets  [n_groups + 1] int32: group g holds the sorted positions
 *            offsets[g] .. offsets[g + 1] - 1             (input)
 *   perm     [n_rows] int32: row at each sorted position, or NULL when the
 *            rows already are in group order              (input)
 *   y        [n_rows][n], row stride y_stride             (output)
 *
 * offsets and perm are the rowptr and perm of zs_build_csr over the rows'
 * group indices.  Groups may be empty.  Rows at positions before offsets[0] or
 * from offsets[n_groups] on belong to no group and get zeros.  Offsets that
 * decrease, or perm entries that repeat, give unspecified rows but no access
 * outside the arrays; perm entries out of range are skipped.
 * The gradient with respect to x is the same call on grad_y with w_transposed
 * flipped and k and n exchanged.
 */
int zs_grouped_mm(const void *x, int64_t x_stride, const void *w,
                  int64_t w_group_stride, int64_t w_stride, int w_transposed,
                  const int32_t *offsets, const int32_t *perm, int64_t n_rows,
                  int64_t n_groups, int64_t k, int64_t n, int dtype, void *y,
                  int64_t y_stride, void *stream);

/*
 * zs_grouped_mm_wgrad -- grad_w[g] = sum over the rows i of group g of
 * x[i]^T grad_y[i], the weight gradient of zs_grouped_mm.
 *
 *   x        [n_rows][k], row stride x_stride             (input)
 *   grad_y   [n_rows][n], row stride gy_stride            (input)
 *   offsets, perm                                         as above
 *   grad_w   [n_groups][k][n] contiguous, of the same dtype, zeros for empty
 *            groups                                       (output)
 *   workspace, workspace_bytes >= zs_grouped_mm_wgrad_workspace_bytes(...),
 *            256-byte aligned device scratch (may be NULL when that is 0).
 *            Long groups are cut into pieces whose fp32 partial sums are kept
 *            there and added in order.
 * The gradient of weights stored [n][k] is the call with x and grad_y (and k
 * and n) exchanged.
 */
size_t zs_grouped_mm_wgrad_workspace_bytes(int64_t n_rows, int64_t n_groups,
                                           int64_t k, int64_t n, int dtype);
int zs_grouped_mm_wgrad(const void *x, int64_t x_stride, const void *grad_y,
                        int64_t gy_stride, const int32_t *offsets,
                        const int32_t *perm, int64_t n_rows, int64_t n_groups,
                        int64_t k, int64_t n, int dtype, void *grad_w,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * zs_grouped_mm_backward -- both gradients of zs_grouped_mm (weights stored
 * [k][n]) in one call: grad_x [n_rows][k] and grad_w [n_groups][k][n], both
 * contiguous, as the two calls above give them up to the order of fp32 sums.
 * Narrow weights (k <= 64, n <= 128, operands on 16 bytes) take one pass that
 * reads grad_y once.  Workspace as zs_grouped_mm_wgrad.
 */
int zs_grouped_mm_backward(const void *grad_y, int64_t gy_stride, const void *x,
                           int64_t x_stride, const void *w,
                           int64_t w_group_stride, int64_t w_stride,
                           const int32_t *offsets, const int32_t *perm,
                           int64_t n_rows, int64_t n_groups, int64_t k,
                           int64_t n, int dtype, void *grad_x, void *grad_w,
                           void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * zs_block_join -- the join of a block's output z with its residual stream x,
 * from the norm behind the block to the norm before the next one:
 *
 *   u = z * (mean(z^2) + eps)^(-1/2) * w_post
 *   y = x + scale * sigmoid(gate) * u
 *   h = y * (mean(y^2) + eps)^(-1/2) * w_pre
 *
 * with means over the c channels of a row.
 *
 *   x, z     [n_rows][c], row strides x_stride, z_stride  (input; z may be
 *            NULL: y = x is then not written, gate, scale and w_post are
 *            ignored, and h is the plain norm of x)
 *   gate     [n_rows][gate_width], row stride gate_stride; gate_width c (a gate
 *            per channel), 1 (a gate per row) or 0 (none: the factor is 1, gate
 *            may be NULL)                                  (input)
 *   scale, w_post [c] fp32                                 (input)
 *   w_pre    [c] fp32, or NULL when no norm follows (h is then not written)
 *   y, h     [n_rows][c] contiguous                        (output)
 * x, z, gate, y and h have the type `dtype`.  h is formed from y before its
 * rounding.  eps > 0.
 */
int zs_block_join(const void *x, int64_t x_stride, const void *z,
                  int64_t z_stride, const void *gate, int64_t gate_stride,
                  int64_t gate_width, const float *scale, const float *w_post,
                  const float *w_pre, int64_t n_rows, int64_t c, float eps,
                  int dtype, void *y, void *h, void *stream);

/*
 * zs_block_join_backward -- gradients of zs_block_join's inputs from those of
 * its outputs; everything else is recomputed from the inputs.
 *
 *   grad_y, grad_h [n_rows][c] contiguous; either may be NULL (zeros)
 *   grad_x, grad_z [n_rows][c], grad_gate [n_rows][gate_width] contiguous
 *            (output; grad_z, grad_gate, grad_scale and grad_w_post are not
 *            written when z is NULL, grad_gate not when gate_width is 0,
 *            grad_w_pre not when w_pre is NULL)
 *   grad_scale, grad_w_post, grad_w_pre [c] fp32           (output)
 *   workspace, workspace_bytes >= zs_block_join_workspace_bytes(n_rows, c),
 *            256-byte aligned device scratch: partial sums of the parameter
 *            gradients, added in a fixed order
 */
size_t zs_block_join_workspace_bytes(int64_t n_rows, int64_t c);
int zs_block_join_backward(const void *grad_y, const void *grad_h,
                           const void *x, int64_t x_stride, const void *z,
                           int64_t z_stride, const void *gate,
                           int64_t gate_stride, int64_t gate_width,
                           const float *scale, const float *w_post,
                           const float *w_pre, int64_t n_rows, int64_t c,
                           float eps, int dtype, void *grad_x, void *grad_z,
                           void *grad_gate, float *grad_scale,
                           float *grad_w_post, float *grad_w_pre,
                           void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * zs_adamw_step -- one AdamW step (decoupled weight decay) over many tensors:
 *
 *   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
 *   p = (1 - lr weight_decay) p
 *       - lr / (1 - beta1^t) m / (sqrt(v) (1 - beta2^t)^(-1/2) + eps)
 *
 * each operation rounded to fp32 in the order written (no fused multiply-add).
 * tensors is a HOST array, read before the call returns.  Parameters are fp32;
 * a gradient is fp32 or bf16; copy, when not NULL, receives the new parameter
 * rounded to bf16 (the working copy of the products).  The states of all
 * tensors lie in one array each: tensor i owns n elements from state_offset, a
 * multiple of ZS_ADAMW_BLOCK, in increasing order and not in one another.
 * Elements between slices are not touched.  Parameters and copies of different
 * tensors must not share memory (not checked here: the host would compare all
 * pairs at every step; the binding's AdamW checks it where an address changed).
 *
 * The config is a host struct too, so a call captured in a HIP graph holds its
 * step: every replay applies that number's bias corrections and rate and, in
 * zs_adamw_step8, adds the same random bits to the same elements, so that a
 * moment which these bits never carry over stays on its code.  A training loop
 * captures its products and gradients and calls the step itself.
 */
typedef struct zs_adamw_tensor {
    float *param;           /* [n], updated in place                          */
    const void *grad;       /* [n], type grad_dtype                           */
    void *copy;             /* [n] bf16 or NULL                               */
    int64_t n;              /* elements, >= 0                                 */
    int64_t state_offset;   /* first element in the state arrays              */
    int32_t grad_dtype;     /* zs_dtype                                       */
    int32_t reserved;       /* 0                                              */
} zs_adamw_tensor;

typedef struct zs_adamw_config {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;           /* t >= 1: the number of this step                */
} zs_adamw_config;

int zs_adamw_step(const zs_adamw_tensor *tensors, int64_t n_tensors,
                  const zs_adamw_config *config, float *m, float *v,
                  int64_t state_elements, void *stream);

/*
 * zs_adamw_step8 -- the same step with m and sqrt(v) held in 8 bits.
 *
 * A block of ZS_ADAMW_BLOCK consecutive state elements shares an fp32 scale,
 * the largest magnitude in it; a value's share t = |value| / scale in [0, 1]
 * is held as a code whose step halves with each power of two:
 *   m_code: sign in bit 7, 7-bit code c; c > 0 stands for the float of bits
 *           (c + 889) << 20, 0 for zero (8 steps a power of two, 15.8 octaves)
 *   v_code: 8-bit code c of sqrt(v); c > 0 stands for the float of bits
 *           (c + 1777) << 19, 0 for zero (16 steps, 15.9 octaves)
 * The top codes stand for 1.  Rounding is stochastic: bits of a hash of the
 * element's index in its slice and (seed + step) mod 2^32 are added below the
 * kept bits, so a moment that changes by less than half a step a time still
 * moves on average.  Codes of sqrt(v) > 0 are at least 1: a positive second
 * moment never becomes zero.  A block whose scale is under 2^-120 becomes
 * zero; one that holds an infinity or NaN decodes to NaN.  Padding elements
 * behind a slice's end, up to the next block, are written as zeros.
 */
int zs_adamw_step8(const zs_adamw_tensor *tensors, int64_t n_tensors,
                   const zs_adamw_config *config, uint8_t *m_code,
                   float *m_scale, uint8_t *v_code, float *v_scale,
                   int64_t state_elements, uint32_t seed, void *stream);

/* The moments that 8-bit states stand for: m and v [state_elements] fp32. */
int zs_adamw_moments8(const uint8_t *m_code, const float *m_scale,
                      const uint8_t *v_code, const float *v_scale,
                      int64_t state_elements, float *m, float *v, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZS_BLOCK_H_ */
