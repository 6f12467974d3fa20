// Declarations shared by the translation units of the grouped products, the
// residual join and AdamW.  Not part of the public ABI (include/zs_block.h).
#pragma once

#include "zs_block.h"
#include "zs_internal.h"

namespace zs {

// Operands of y[i] = x[i] op(w[g(i)]) on checked arguments.
struct GmmArgs {
    const void* x;
    const void* w;
    void* y;
    const int32_t* offsets;
    const int32_t* perm;
    int64_t ldx, ldw, w_group, ldy;   // strides in elements
    int64_t n_rows, n_groups;
    int k, n;
};

hipError_t launch_gmm(const GmmArgs& a, bool bf16, bool w_transposed, hipStream_t stream);

// Operands of grad_w[g] = x_g^T grad_y_g; partial: fp32 sums of row pieces.
struct WgradArgs {
    const void* x;
    const void* gy;
    void* gw;
    float* partial;
    const int32_t* offsets;
    const int32_t* perm;
    int64_t ldx, ldg;
    int64_t n_rows, n_groups;
    int64_t piece;   // rows of a piece; above n_rows: groups are never cut
    int k, n;
    // where both_gradients() says so: grad_x [n_rows][k] too, from w [k][n]
    const void* w;
    void* gx;
    int64_t ldw, w_group;
};
// Whether one kernel forms both gradients: the weights are one tile.
bool both_gradients(const WgradArgs& a, bool bf16);

// How the weight gradient is cut: rows per piece and the bytes its partial
// sums take (0: no group is cut).
struct WgradPlan {
    int64_t piece;
    size_t bytes;
};
WgradPlan plan_wgrad(int64_t n_rows, int64_t n_groups, int64_t k, int64_t n, bool bf16);
hipError_t launch_wgrad(const WgradArgs& a, bool bf16, hipStream_t stream);

struct JoinArgs {
    const void* x;
    const void* z;
    const void* gate;
    int64_t ldx, ldz, ldg;
    int64_t gate_width;
    const float *scale, *w_post, *w_pre;
    int64_t n_rows;
    int c;
    float eps;
    // forward
    void *y, *h;
    // backward
    const void *gy, *gh;
    void *gx, *gz, *ggate;
    float *gscale, *gpost, *gpre;
    float* partial;
};
hipError_t launch_join(const JoinArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_join_backward(const JoinArgs& a, bool bf16, hipStream_t stream);
size_t join_workspace(int64_t n_rows, int64_t c);

// Constants of one AdamW step, rounded to fp32 once on the host.
struct AdamwConst {
    float beta1, one_beta1, beta2, one_beta2, keep, root_scale, eps, rate;
};
hipError_t launch_adamw(const zs_adamw_tensor* tensors, int64_t n_tensors, AdamwConst c, float* m,
                        float* v, hipStream_t stream);
hipError_t launch_adamw8(const zs_adamw_tensor* tensors, int64_t n_tensors, AdamwConst c,
                         uint8_t* mc, float* ms, uint8_t* vc, float* vs, uint32_t key,
                         hipStream_t stream);
hipError_t launch_moments8(const uint8_t* mc, const float* ms, const uint8_t* vc, const float* vs,
                           int64_t n, float* m, float* v, hipStream_t stream);

}  // namespace zs
