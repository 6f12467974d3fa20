// Declarations shared by the translation units of the lookup, the layer norm, the
// router and the weighted sum.  Not part of the public ABI (include/zs_layers.h).
#pragma once

#include "zs_internal.h"
#include "zs_layers.h"

namespace zs {

struct EmbedArgs {
    const void* table;
    int64_t ldt;
    const int64_t* index;
    int64_t n_rows, n_entries;
    int c;
    float scale;
    void* y;
};
hipError_t launch_embed(const EmbedArgs& a, bool bf16, hipStream_t stream);

struct EmbedGradArgs {
    const void* gy;
    int64_t ldg;
    const int64_t* index;
    const int32_t *offsets, *perm;
    int64_t n_rows, n_entries;
    int c;
    float scale;
    void* grad;
    void* workspace;
};
// Bytes of the sums that the workgroups leave to each other (0: a single workgroup).
size_t embed_grad_workspace(int64_t n_rows, int64_t c, bool bf16);
hipError_t launch_embed_grad(const EmbedGradArgs& a, bool bf16, hipStream_t stream);

struct NormArgs {
    const void* x;
    int64_t ldx;
    const float *w, *b;
    int64_t n_rows;
    int c;
    float eps;
    void* y;   // forward
    // backward
    const void* gy;
    int64_t ldg;
    void* gx;
    float *gw, *gb;
    float* partial;
};
hipError_t launch_layer_norm(const NormArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_layer_norm_backward(const NormArgs& a, bool bf16, hipStream_t stream);
size_t layer_norm_workspace(int64_t n_rows, int64_t c);

struct RouteArgs {
    const void* x;
    int64_t ldx;
    const float* bias;
    zs_router r;
    int64_t n_rows;
    int n;   // experts
    // forward
    float* weight;
    int64_t* expert;
    // backward
    const float* gw;
    const int64_t* chosen;
    void* gx;
};
hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t stream);

struct CombineArgs {
    const void* z;
    int64_t ldz;
    const float* weight;
    int64_t n_rows;
    int k, c;
    void* y;   // forward
    // backward
    const void* gy;
    int64_t ldg;
    void* gz;
    float* gw;
};
hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_combine_backward(const CombineArgs& a, bool bf16, hipStream_t stream);

}  // namespace zs
