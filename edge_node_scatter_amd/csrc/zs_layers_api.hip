// C ABI of the lookup, the layer norm, the router and the weighted sum (declared
// in include/zs_layers.h): argument checks on the host, then kernel dispatch.
// Every check runs before the first HIP call, so a rejected call leaves device
// state untouched.
#include "zs_layers.h"

#include <cmath>

#include "zs_check.h"
#include "zs_layers_internal.h"

using namespace zs::check;

namespace {

bool width_ok(int64_t c) { return c >= 1 && c <= ZS_MAX_LAYER_WIDTH; }
bool rows_ok(int64_t n) { return n >= 0 && n <= ZS_MAX_EDGES; }

}  // namespace

extern "C" {

int zs_embedding(const void* table, int64_t table_stride, const int64_t* index, int64_t n_rows,
                 int64_t n_entries, int64_t c, float scale, int dtype, void* y, void* stream) {
    if (!rows_ok(n_rows) || n_entries < 1 || n_entries > ZS_MAX_NODES || !width_ok(c) ||
        table_stride < 0)
        return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t et = extent(n_entries, table_stride, c);
    if (et < 0) return ZS_ERR_SHAPE;
    if (n_rows == 0) return ZS_OK;
    if (!table || !index || !y) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(table, es) || !aligned(y, es) || !aligned(index, 8)) return ZS_ERR_UNSUPPORTED;
    const Range out = span(y, n_rows * c * es);
    const Range ins[] = {span(table, et * es), span(index, n_rows * 8)};
    if (aliased(&out, 1, ins, 2)) return ZS_ERR_ALIAS;
    const zs::EmbedArgs a{table, table_stride, index, n_rows, n_entries, int(c), scale, y};
    return hip_status(zs::launch_embed(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

size_t zs_embedding_backward_workspace_bytes(int64_t n_rows, int64_t c, int dtype) {
    if (!rows_ok(n_rows) || !width_ok(c) || !dtype_ok(dtype)) return 0;
    return zs::embed_grad_workspace(n_rows, c, dtype == ZS_BF16);
}

int zs_embedding_backward(const void* grad_y, int64_t gy_stride, const int64_t* index,
                          const int32_t* offsets, const int32_t* perm, int64_t n_rows,
                          int64_t n_entries, int64_t c, float scale, int dtype, void* grad_table,
                          void* workspace, size_t workspace_bytes, void* stream) {
    if (!rows_ok(n_rows) || n_entries < 1 || n_entries > ZS_MAX_NODES || !width_ok(c) ||
        gy_stride < 0)
        return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t eg = extent(n_rows, gy_stride, c);
    const int64_t es = size_of(dtype);
    if (eg < 0) return ZS_ERR_SHAPE;
    if (!offsets || !grad_table || (n_rows > 0 && (!grad_y || !index))) return ZS_ERR_NULL;
    if (!aligned(grad_y, es) || !aligned(grad_table, es) || !aligned(index, 8) ||
        !aligned(offsets, 4) || !aligned(perm, 4))
        return ZS_ERR_UNSUPPORTED;
    const size_t need = zs::embed_grad_workspace(n_rows, c, dtype == ZS_BF16);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return ZS_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return ZS_ERR_UNSUPPORTED;
    }
    const Range outs[] = {span(grad_table, n_entries * c * es),
                          span(need ? workspace : nullptr, int64_t(need))};
    const Range ins[] = {span(grad_y, eg * es), span(index, n_rows * 8),
                         span(offsets, (n_entries + 1) * 4), span(perm, n_rows * 4)};
    if (aliased(outs, 2, ins, 4)) return ZS_ERR_ALIAS;
    const zs::EmbedGradArgs a{grad_y, gy_stride, index,  offsets,    perm,     n_rows,
                              n_entries, int(c), scale, grad_table, workspace};
    return hip_status(
        zs::launch_embed_grad(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

int zs_layer_norm(const void* x, int64_t x_stride, const float* w, const float* b, int64_t n_rows,
                  int64_t c, float eps, int dtype, void* y, void* stream) {
    if (!rows_ok(n_rows) || !width_ok(c) || x_stride < 0 || !(eps > 0.0f) || !std::isfinite(eps))
        return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t ex = extent(n_rows, x_stride, c);
    if (ex < 0) return ZS_ERR_SHAPE;
    if (n_rows == 0) return ZS_OK;
    if (!x || !w || !y) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(w, 4) || !aligned(b, 4))
        return ZS_ERR_UNSUPPORTED;
    const Range out = span(y, n_rows * c * es);
    const Range ins[] = {span(x, ex * es), span(w, c * 4), span(b, c * 4)};
    if (aliased(&out, 1, ins, 3)) return ZS_ERR_ALIAS;
    zs::NormArgs a{};
    a.x = x, a.ldx = x_stride, a.w = w, a.b = b, a.n_rows = n_rows, a.c = int(c), a.eps = eps;
    a.y = y;
    return hip_status(zs::launch_layer_norm(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

size_t zs_layer_norm_workspace_bytes(int64_t n_rows, int64_t c) {
    if (!rows_ok(n_rows) || !width_ok(c)) return 0;
    return zs::layer_norm_workspace(n_rows, c);
}

int zs_layer_norm_backward(const void* grad_y, int64_t gy_stride, const void* x, int64_t x_stride,
                           const float* w, int64_t n_rows, int64_t c, float eps, int dtype,
                           void* grad_x, float* grad_w, float* grad_b, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (!rows_ok(n_rows) || !width_ok(c) || x_stride < 0 || gy_stride < 0 || !(eps > 0.0f) ||
        !std::isfinite(eps))
        return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t ex = extent(n_rows, x_stride, c), eg = extent(n_rows, gy_stride, c);
    if (ex < 0 || eg < 0) return ZS_ERR_SHAPE;
    if (!w || !grad_w || (n_rows > 0 && (!grad_y || !x || !grad_x))) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(grad_y, es) || !aligned(x, es) || !aligned(grad_x, es) || !aligned(w, 4) ||
        !aligned(grad_w, 4) || !aligned(grad_b, 4))
        return ZS_ERR_UNSUPPORTED;
    const size_t need = zs::layer_norm_workspace(n_rows, c);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return ZS_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return ZS_ERR_UNSUPPORTED;
    }
    const Range outs[] = {span(grad_x, n_rows * c * es), span(grad_w, c * 4), span(grad_b, c * 4),
                          span(need ? workspace : nullptr, int64_t(need))};
    const Range ins[] = {span(grad_y, eg * es), span(x, ex * es), span(w, c * 4)};
    if (aliased(outs, 4, ins, 3)) return ZS_ERR_ALIAS;
    zs::NormArgs a{};
    a.x = x, a.ldx = x_stride, a.w = w, a.n_rows = n_rows, a.c = int(c), a.eps = eps;
    a.gy = grad_y, a.ldg = gy_stride, a.gx = grad_x, a.gw = grad_w, a.gb = grad_b;
    a.partial = static_cast<float*>(workspace);
    return hip_status(
        zs::launch_layer_norm_backward(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Checks shared by the router's two directions.
int router_ok(const zs_router* r, int64_t n_rows, int64_t n_experts, int64_t stride) {
    if (!r) return ZS_ERR_NULL;
    if (!rows_ok(n_rows) || n_experts < 1 || n_experts > ZS_MAX_EXPERTS || stride < 0)
        return ZS_ERR_SHAPE;
    if (r->groups < 1 || r->groups > ZS_MAX_EXPERT_GROUPS || n_experts % r->groups != 0 ||
        r->top_groups < 1 || r->top_groups > r->groups || r->k < 1 || r->k > ZS_MAX_SLOTS ||
        r->k > n_experts / r->groups * r->top_groups || r->best < 1 || r->best > 2 ||
        r->sigmoid < 0 || r->sigmoid > 1 || r->renormalise < 0 || r->renormalise > 1 ||
        !std::isfinite(r->scale))
        return ZS_ERR_SHAPE;
    return n_rows * r->k > ZS_MAX_EDGES ? ZS_ERR_SHAPE : ZS_OK;
}

}  // namespace

extern "C" {

int zs_route(const void* logits, int64_t logits_stride, const float* bias, const zs_router* router,
             int64_t n_rows, int64_t n_experts, int dtype, float* weight, int64_t* expert,
             void* stream) {
    const int st = router_ok(router, n_rows, n_experts, logits_stride);
    if (st != ZS_OK) return st;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t ex = extent(n_rows, logits_stride, n_experts);
    if (ex < 0) return ZS_ERR_SHAPE;
    if (n_rows == 0) return ZS_OK;
    if (!logits || !weight || !expert) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype), slots = n_rows * router->k;
    if (!aligned(logits, es) || !aligned(bias, 4) || !aligned(weight, 4) || !aligned(expert, 8))
        return ZS_ERR_UNSUPPORTED;
    const Range outs[] = {span(weight, slots * 4), span(expert, slots * 8)};
    const Range ins[] = {span(logits, ex * es), span(bias, n_experts * 4)};
    if (aliased(outs, 2, ins, 2)) return ZS_ERR_ALIAS;
    zs::RouteArgs a{};
    a.x = logits, a.ldx = logits_stride, a.bias = bias, a.r = *router;
    a.n_rows = n_rows, a.n = int(n_experts), a.weight = weight, a.expert = expert;
    return hip_status(zs::launch_route(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

int zs_route_backward(const float* grad_weight, const void* logits, int64_t logits_stride,
                      const int64_t* expert, const zs_router* router, int64_t n_rows,
                      int64_t n_experts, int dtype, void* grad_logits, void* stream) {
    const int st = router_ok(router, n_rows, n_experts, logits_stride);
    if (st != ZS_OK) return st;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t ex = extent(n_rows, logits_stride, n_experts);
    if (ex < 0) return ZS_ERR_SHAPE;
    if (n_rows == 0) return ZS_OK;
    if (!grad_weight || !logits || !expert || !grad_logits) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype), slots = n_rows * router->k;
    if (!aligned(logits, es) || !aligned(grad_logits, es) || !aligned(grad_weight, 4) ||
        !aligned(expert, 8))
        return ZS_ERR_UNSUPPORTED;
    const Range out = span(grad_logits, n_rows * n_experts * es);
    const Range ins[] = {span(grad_weight, slots * 4), span(logits, ex * es),
                         span(expert, slots * 8)};
    if (aliased(&out, 1, ins, 3)) return ZS_ERR_ALIAS;
    zs::RouteArgs a{};
    a.x = logits, a.ldx = logits_stride, a.r = *router, a.n_rows = n_rows, a.n = int(n_experts);
    a.gw = grad_weight, a.chosen = expert, a.gx = grad_logits;
    return hip_status(
        zs::launch_route_backward(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

int combine_ok(int64_t n_rows, int64_t k, int64_t c, int64_t z_stride) {
    if (!rows_ok(n_rows) || k < 1 || k > ZS_MAX_SLOTS || !rows_ok(n_rows * k) || !width_ok(c) ||
        z_stride < 0)
        return ZS_ERR_SHAPE;
    return ZS_OK;
}

}  // namespace

extern "C" {

int zs_combine(const void* z, int64_t z_stride, const float* weight, int64_t n_rows, int64_t k,
               int64_t c, int dtype, void* y, void* stream) {
    const int st = combine_ok(n_rows, k, c, z_stride);
    if (st != ZS_OK) return st;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t ez = extent(n_rows * k, z_stride, c);
    if (ez < 0) return ZS_ERR_SHAPE;
    if (n_rows == 0) return ZS_OK;
    if (!z || !weight || !y) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(z, es) || !aligned(y, es) || !aligned(weight, 4)) return ZS_ERR_UNSUPPORTED;
    const Range out = span(y, n_rows * c * es);
    const Range ins[] = {span(z, ez * es), span(weight, n_rows * k * 4)};
    if (aliased(&out, 1, ins, 2)) return ZS_ERR_ALIAS;
    zs::CombineArgs a{};
    a.z = z, a.ldz = z_stride, a.weight = weight, a.n_rows = n_rows, a.k = int(k), a.c = int(c);
    a.y = y;
    return hip_status(zs::launch_combine(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

int zs_combine_backward(const void* grad_y, int64_t gy_stride, const void* z, int64_t z_stride,
                        const float* weight, int64_t n_rows, int64_t k, int64_t c, int dtype,
                        void* grad_z, float* grad_weight, void* stream) {
    const int st = combine_ok(n_rows, k, c, z_stride);
    if (st != ZS_OK) return st;
    if (gy_stride < 0) return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t ez = extent(n_rows * k, z_stride, c), eg = extent(n_rows, gy_stride, c);
    if (ez < 0 || eg < 0) return ZS_ERR_SHAPE;
    if (n_rows == 0) return ZS_OK;
    if (!grad_y || !z || !weight || !grad_z || !grad_weight) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(grad_y, es) || !aligned(z, es) || !aligned(grad_z, es) || !aligned(weight, 4) ||
        !aligned(grad_weight, 4))
        return ZS_ERR_UNSUPPORTED;
    const Range outs[] = {span(grad_z, n_rows * k * c * es), span(grad_weight, n_rows * k * 4)};
    const Range ins[] = {span(grad_y, eg * es), span(z, ez * es), span(weight, n_rows * k * 4)};
    if (aliased(outs, 2, ins, 3)) return ZS_ERR_ALIAS;
    zs::CombineArgs a{};
    a.z = z, a.ldz = z_stride, a.weight = weight, a.n_rows = n_rows, a.k = int(k), a.c = int(c);
    a.gy = grad_y, a.ldg = gy_stride, a.gz = grad_z, a.gw = grad_weight;
    return hip_status(
        zs::launch_combine_backward(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
