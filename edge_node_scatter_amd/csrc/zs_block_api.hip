// C ABI of the grouped products, the residual join and AdamW (declared in
// include/zs_block.h): argument checks on the host, then kernel dispatch.
// Every check runs before the first HIP call, so a rejected call leaves device
// state untouched.
#include "zs_block.h"

#include <cmath>

#include "zs_block_internal.h"
#include "zs_check.h"

using namespace zs::check;

namespace {

bool mm_sizes_ok(int64_t n_rows, int64_t n_groups, int64_t k, int64_t n) {
    return n_rows >= 0 && n_rows <= ZS_MAX_EDGES && n_groups >= 1 && n_groups <= ZS_MAX_GROUPS &&
           k >= 1 && k <= ZS_MAX_WIDTH && n >= 1 && n <= ZS_MAX_WIDTH;
}

}  // namespace

extern "C" {

int zs_grouped_mm(const void* x, int64_t x_stride, const void* w, int64_t w_group_stride,
                  int64_t w_stride, int w_transposed, const int32_t* offsets, const int32_t* perm,
                  int64_t n_rows, int64_t n_groups, int64_t k, int64_t n, int dtype, void* y,
                  int64_t y_stride, void* stream) {
    if (!mm_sizes_ok(n_rows, n_groups, k, n)) return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    const int64_t w_rows = w_transposed ? n : k, w_cols = w_transposed ? k : n;
    if (x_stride < 0 || y_stride < n || w_stride < 0 || w_group_stride < 0)
        return ZS_ERR_SHAPE;
    const int64_t ex = extent(n_rows, x_stride, k), ey = extent(n_rows, y_stride, n),
                  eg = extent(w_rows, w_stride, w_cols);
    const int64_t ew = eg < 0 ? -1 : extent(n_groups, w_group_stride, eg);
    if (ex < 0 || ey < 0 || ew < 0) return ZS_ERR_SHAPE;
    if (n_rows == 0) return ZS_OK;
    if (!x || !w || !offsets || !y) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(x, es) || !aligned(w, es) || !aligned(y, es) || !aligned(offsets, 4) ||
        !aligned(perm, 4))
        return ZS_ERR_UNSUPPORTED;
    const Range out = span(y, ey * es);
    const Range ins[] = {span(x, ex * es), span(w, ew * es), span(offsets, (n_groups + 1) * 4),
                         span(perm, n_rows * 4)};
    if (aliased(&out, 1, ins, 4)) return ZS_ERR_ALIAS;
    const zs::GmmArgs a{x,        w,       y,        offsets, perm,     x_stride, w_stride,
                        w_group_stride, y_stride, n_rows,  n_groups, int(k),   int(n)};
    return hip_status(zs::launch_gmm(a, dtype == ZS_BF16, w_transposed != 0,
                                     static_cast<hipStream_t>(stream)));
}

size_t zs_grouped_mm_wgrad_workspace_bytes(int64_t n_rows, int64_t n_groups, int64_t k, int64_t n,
                                           int dtype) {
    if (!mm_sizes_ok(n_rows, n_groups, k, n) || !dtype_ok(dtype)) return 0;
    return zs::plan_wgrad(n_rows, n_groups, k, n, dtype == ZS_BF16).bytes;
}

int zs_grouped_mm_wgrad(const void* x, int64_t x_stride, const void* grad_y, int64_t gy_stride,
                        const int32_t* offsets, const int32_t* perm, int64_t n_rows,
                        int64_t n_groups, int64_t k, int64_t n, int dtype, void* grad_w,
                        void* workspace, size_t workspace_bytes, void* stream) {
    if (!mm_sizes_ok(n_rows, n_groups, k, n)) return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    if (x_stride < 0 || gy_stride < 0) return ZS_ERR_SHAPE;
    const int64_t ex = extent(n_rows, x_stride, k), eg = extent(n_rows, gy_stride, n);
    if (ex < 0 || eg < 0) return ZS_ERR_SHAPE;
    if (!offsets || !grad_w || (n_rows > 0 && (!x || !grad_y))) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(x, es) || !aligned(grad_y, es) || !aligned(grad_w, es) || !aligned(offsets, 4) ||
        !aligned(perm, 4))
        return ZS_ERR_UNSUPPORTED;
    const zs::WgradPlan plan = zs::plan_wgrad(n_rows, n_groups, k, n, dtype == ZS_BF16);
    if (plan.bytes > 0) {
        if (!workspace || workspace_bytes < plan.bytes) return ZS_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return ZS_ERR_UNSUPPORTED;
    }
    const Range outs[] = {span(grad_w, n_groups * k * n * es),
                          span(plan.bytes ? workspace : nullptr, int64_t(plan.bytes))};
    const Range ins[] = {span(x, ex * es), span(grad_y, eg * es), span(offsets, (n_groups + 1) * 4),
                         span(perm, n_rows * 4)};
    if (aliased(outs, 2, ins, 4)) return ZS_ERR_ALIAS;
    const zs::WgradArgs a{x,        grad_y,    grad_w, static_cast<float*>(workspace),
                          offsets,  perm,      x_stride, gy_stride,
                          n_rows,   n_groups,  plan.piece, int(k), int(n), nullptr, nullptr, 0, 0};
    return hip_status(zs::launch_wgrad(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

int zs_grouped_mm_backward(const void* grad_y, int64_t gy_stride, const void* x, int64_t x_stride,
                           const void* w, int64_t w_group_stride, int64_t w_stride,
                           const int32_t* offsets, const int32_t* perm, int64_t n_rows,
                           int64_t n_groups, int64_t k, int64_t n, int dtype, void* grad_x,
                           void* grad_w, void* workspace, size_t workspace_bytes, void* stream) {
    if (!mm_sizes_ok(n_rows, n_groups, k, n)) return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    if (x_stride < 0 || gy_stride < 0 || w_stride < 0 || w_group_stride < 0) return ZS_ERR_SHAPE;
    const int64_t ex = extent(n_rows, x_stride, k), eg = extent(n_rows, gy_stride, n),
                  e1 = extent(k, w_stride, n);
    const int64_t ew = e1 < 0 ? -1 : extent(n_groups, w_group_stride, e1);
    if (ex < 0 || eg < 0 || ew < 0) return ZS_ERR_SHAPE;
    if (!offsets || !grad_w || (n_rows > 0 && (!x || !grad_y || !w || !grad_x))) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype);
    if (!aligned(x, es) || !aligned(grad_y, es) || !aligned(w, es) || !aligned(grad_x, es) ||
        !aligned(grad_w, es) || !aligned(offsets, 4) || !aligned(perm, 4))
        return ZS_ERR_UNSUPPORTED;
    const zs::WgradPlan plan = zs::plan_wgrad(n_rows, n_groups, k, n, dtype == ZS_BF16);
    if (plan.bytes > 0) {
        if (!workspace || workspace_bytes < plan.bytes) return ZS_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return ZS_ERR_UNSUPPORTED;
    }
    const Range outs[] = {span(grad_w, n_groups * k * n * es), span(grad_x, n_rows * k * es),
                          span(plan.bytes ? workspace : nullptr, int64_t(plan.bytes))};
    const Range ins[] = {span(x, ex * es), span(grad_y, eg * es), span(w, ew * es),
                         span(offsets, (n_groups + 1) * 4), span(perm, n_rows * 4)};
    if (aliased(outs, 3, ins, 5)) return ZS_ERR_ALIAS;
    const bool bf16 = dtype == ZS_BF16;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    zs::WgradArgs a{x,      grad_y,   grad_w,     static_cast<float*>(workspace),
                    offsets, perm,    x_stride,   gy_stride,
                    n_rows, n_groups, plan.piece, int(k), int(n), w, grad_x, w_stride,
                    w_group_stride};
    if (n_rows == 0 || !zs::both_gradients(a, bf16)) {
        a.gx = nullptr;
        if (n_rows > 0) {
            const zs::GmmArgs g{grad_y,  w,        grad_x,         offsets, perm,     gy_stride,
                                w_stride, w_group_stride, k, n_rows,  n_groups, int(n), int(k)};
            const hipError_t err = zs::launch_gmm(g, bf16, true, s);
            if (err != hipSuccess) return ZS_ERR_HIP;
        }
    }
    return hip_status(zs::launch_wgrad(a, bf16, s));
}

}  // extern "C"

namespace {

// Checks shared by the join's two directions.  On ZS_OK fills the byte extents
// of the strided inputs.
int join_inputs(const void* x, int64_t x_stride, const void* z, int64_t z_stride, const void* gate,
                int64_t gate_stride, int64_t gate_width, const float* scale, const float* w_post,
                const float* w_pre, int64_t n_rows, int64_t c, float eps, int dtype,
                int64_t (&bytes)[3]) {
    if (n_rows < 0 || n_rows > ZS_MAX_EDGES || c < 1 || c > ZS_MAX_JOIN_WIDTH) return ZS_ERR_SHAPE;
    if (!dtype_ok(dtype)) return ZS_ERR_UNSUPPORTED;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return ZS_ERR_SHAPE;
    if (gate_width != 0 && gate_width != 1 && gate_width != c) return ZS_ERR_SHAPE;
    if (x_stride < 0 || (z && z_stride < 0) || (z && gate_width && gate_stride < 0))
        return ZS_ERR_SHAPE;
    const int64_t es = size_of(dtype);
    const int64_t ex = extent(n_rows, x_stride, c), ez = z ? extent(n_rows, z_stride, c) : 0,
                  eg = z && gate_width ? extent(n_rows, gate_stride, gate_width) : 0;
    if (ex < 0 || ez < 0 || eg < 0) return ZS_ERR_SHAPE;
    if (n_rows > 0 && (!x || (z && gate_width && !gate))) return ZS_ERR_NULL;
    if (z && (!scale || !w_post)) return ZS_ERR_NULL;
    if (!z && !w_pre) return ZS_ERR_NULL;
    if (!aligned(x, es) || !aligned(z, es) || !aligned(gate, es) || !aligned(scale, 4) ||
        !aligned(w_post, 4) || !aligned(w_pre, 4))
        return ZS_ERR_UNSUPPORTED;
    bytes[0] = ex * es;
    bytes[1] = ez * es;
    bytes[2] = eg * es;
    return ZS_OK;
}

}  // namespace

extern "C" {

int zs_block_join(const void* x, int64_t x_stride, const void* z, int64_t z_stride,
                  const void* gate, int64_t gate_stride, int64_t gate_width, const float* scale,
                  const float* w_post, const float* w_pre, int64_t n_rows, int64_t c, float eps,
                  int dtype, void* y, void* h, void* stream) {
    int64_t b[3];
    const int st = join_inputs(x, x_stride, z, z_stride, gate, gate_stride, gate_width, scale,
                               w_post, w_pre, n_rows, c, eps, dtype, b);
    if (st != ZS_OK) return st;
    if (n_rows == 0) return ZS_OK;
    if ((z && !y) || (w_pre && !h)) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype), dense = n_rows * c * es;
    if (!aligned(y, es) || !aligned(h, es)) return ZS_ERR_UNSUPPORTED;
    if (!z) y = nullptr, gate_width = 0;
    if (!w_pre) h = nullptr;
    if (!gate_width) gate = nullptr;
    const Range outs[] = {span(y, dense), span(h, dense)};
    const Range ins[] = {span(x, b[0]), span(z, b[1]), span(gate, b[2]),
                         span(z ? scale : nullptr, c * 4), span(z ? w_post : nullptr, c * 4),
                         span(w_pre, c * 4)};
    if (aliased(outs, 2, ins, 6)) return ZS_ERR_ALIAS;
    zs::JoinArgs a{};
    a.x = x, a.z = z, a.gate = gate;
    a.ldx = x_stride, a.ldz = z_stride, a.ldg = gate_stride, a.gate_width = gate_width;
    a.scale = scale, a.w_post = w_post, a.w_pre = w_pre;
    a.n_rows = n_rows, a.c = int(c), a.eps = eps;
    a.y = y, a.h = h;
    return hip_status(zs::launch_join(a, dtype == ZS_BF16, static_cast<hipStream_t>(stream)));
}

size_t zs_block_join_workspace_bytes(int64_t n_rows, int64_t c) {
    if (n_rows < 0 || n_rows > ZS_MAX_EDGES || c < 1 || c > ZS_MAX_JOIN_WIDTH) return 0;
    return zs::join_workspace(n_rows, c);
}

int zs_block_join_backward(const void* grad_y, const void* grad_h, const void* x, int64_t x_stride,
                           const void* z, int64_t z_stride, const void* gate, int64_t gate_stride,
                           int64_t gate_width, const float* scale, const float* w_post,
                           const float* w_pre, int64_t n_rows, int64_t c, float eps, int dtype,
                           void* grad_x, void* grad_z, void* grad_gate, float* grad_scale,
                           float* grad_w_post, float* grad_w_pre, void* workspace,
                           size_t workspace_bytes, void* stream) {
    int64_t b[3];
    const int st = join_inputs(x, x_stride, z, z_stride, gate, gate_stride, gate_width, scale,
                               w_post, w_pre, n_rows, c, eps, dtype, b);
    if (st != ZS_OK) return st;
    if (!z) gate_width = 0;
    if (!gate_width) gate = nullptr;
    if ((z && (!grad_scale || !grad_w_post)) || (w_pre && !grad_w_pre)) return ZS_ERR_NULL;
    if (n_rows > 0 && (!grad_x || (z && !grad_z) || (gate_width && !grad_gate))) return ZS_ERR_NULL;
    const int64_t es = size_of(dtype), dense = n_rows * c * es;
    if (!aligned(grad_y, es) || !aligned(grad_h, es) || !aligned(grad_x, es) ||
        !aligned(grad_z, es) || !aligned(grad_gate, es) || !aligned(grad_scale, 4) ||
        !aligned(grad_w_post, 4) || !aligned(grad_w_pre, 4))
        return ZS_ERR_UNSUPPORTED;
    const size_t need = zs::join_workspace(n_rows, c);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return ZS_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return ZS_ERR_UNSUPPORTED;
    }
    if (!z) grad_z = nullptr, grad_scale = grad_w_post = nullptr;
    if (!gate_width) grad_gate = nullptr;
    if (!w_pre) grad_w_pre = nullptr, grad_h = nullptr;
    const Range outs[] = {span(grad_x, dense), span(grad_z, dense),
                          span(grad_gate, n_rows * gate_width * es), span(grad_scale, c * 4),
                          span(grad_w_post, c * 4), span(grad_w_pre, c * 4),
                          span(need ? workspace : nullptr, int64_t(need))};
    const Range ins[] = {span(x, b[0]), span(z, b[1]), span(gate, b[2]), span(grad_y, dense),
                         span(grad_h, dense), span(z ? scale : nullptr, c * 4),
                         span(z ? w_post : nullptr, c * 4), span(w_pre, c * 4)};
    if (aliased(outs, 7, ins, 8)) return ZS_ERR_ALIAS;
    zs::JoinArgs a{};
    a.x = x, a.z = z, a.gate = gate;
    a.ldx = x_stride, a.ldz = z_stride, a.ldg = gate_stride, a.gate_width = gate_width;
    a.scale = scale, a.w_post = w_post, a.w_pre = w_pre;
    a.n_rows = n_rows, a.c = int(c), a.eps = eps;
    a.gy = grad_y, a.gh = grad_h, a.gx = grad_x, a.gz = grad_z, a.ggate = grad_gate;
    a.gscale = grad_scale, a.gpost = grad_w_post, a.gpre = grad_w_pre;
    a.partial = static_cast<float*>(workspace);
    return hip_status(zs::launch_join_backward(a, dtype == ZS_BF16,
                                               static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

bool finite_in(double v, double lo, double hi) { return v >= lo && v <= hi; }

// Checks of a step's tensors against each other and the state arrays: every
// slice inside the state, starting on a block, and no two slices (up to the
// end of their last block) in one another.
int adamw_tensors(const zs_adamw_tensor* t, int64_t n_tensors, const zs_adamw_config* c,
                  int64_t state_elements) {
    if (n_tensors < 0 || n_tensors > (1 << 20) || state_elements < 0 ||
        state_elements > kMaxExtent / 8)
        return ZS_ERR_SHAPE;
    if (!c || (n_tensors > 0 && !t)) return ZS_ERR_NULL;
    if (!finite_in(c->lr, 0.0, 1e30) || !(c->beta1 >= 0.0 && c->beta1 < 1.0) ||
        !(c->beta2 >= 0.0 && c->beta2 < 1.0) || !finite_in(c->eps, 0.0, 1e30) ||
        !finite_in(c->weight_decay, 0.0, 1e30) || c->step < 1)
        return ZS_ERR_SHAPE;
    int64_t last = 0;   // slices come in increasing order, so one pass finds overlaps
    for (int64_t i = 0; i < n_tensors; ++i) {
        if (t[i].n < 0 || t[i].n > state_elements || t[i].state_offset < 0 ||
            t[i].state_offset % ZS_ADAMW_BLOCK != 0 || t[i].state_offset < last)
            return ZS_ERR_SHAPE;
        last = t[i].state_offset + (t[i].n + ZS_ADAMW_BLOCK - 1) / ZS_ADAMW_BLOCK * ZS_ADAMW_BLOCK;
        if (last > state_elements) return ZS_ERR_SHAPE;
        if (t[i].n == 0) continue;
        if (!dtype_ok(t[i].grad_dtype) || t[i].reserved != 0) return ZS_ERR_UNSUPPORTED;
        if (!t[i].param || !t[i].grad) return ZS_ERR_NULL;
        if (!aligned(t[i].param, 4) || !aligned(t[i].grad, size_of(t[i].grad_dtype)) ||
            !aligned(t[i].copy, 2))
            return ZS_ERR_UNSUPPORTED;
        const Range outs[] = {span(t[i].param, t[i].n * 4), span(t[i].copy, t[i].n * 2)};
        const Range in = span(t[i].grad, t[i].n * size_of(t[i].grad_dtype));
        if (aliased(outs, 2, &in, 1)) return ZS_ERR_ALIAS;
    }
    return ZS_OK;
}

// Whether a tensor's arrays overlap a state array.
bool meets_state(const zs_adamw_tensor* t, int64_t n_tensors, const Range* states, int n_states) {
    for (int64_t i = 0; i < n_tensors; ++i) {
        if (t[i].n == 0) continue;
        const Range own[] = {span(t[i].param, t[i].n * 4), span(t[i].copy, t[i].n * 2),
                             span(t[i].grad, t[i].n * size_of(t[i].grad_dtype))};
        for (const Range& r : own)
            for (int j = 0; j < n_states; ++j)
                if (overlap(r, states[j])) return true;
    }
    return false;
}

zs::AdamwConst constants(const zs_adamw_config& c) {
    zs::AdamwConst k;
    k.beta1 = float(c.beta1), k.one_beta1 = float(1.0 - c.beta1);
    k.beta2 = float(c.beta2), k.one_beta2 = float(1.0 - c.beta2);
    k.keep = float(1.0 - c.lr * c.weight_decay);
    k.root_scale = float(std::pow(1.0 - std::pow(c.beta2, double(c.step)), -0.5));
    k.eps = float(c.eps);
    k.rate = float(c.lr / (1.0 - std::pow(c.beta1, double(c.step))));
    return k;
}

}  // namespace

extern "C" {

int zs_adamw_step(const zs_adamw_tensor* tensors, int64_t n_tensors, const zs_adamw_config* config,
                  float* m, float* v, int64_t state_elements, void* stream) {
    const int st = adamw_tensors(tensors, n_tensors, config, state_elements);
    if (st != ZS_OK) return st;
    if (state_elements == 0 || n_tensors == 0) return ZS_OK;
    if (!m || !v) return ZS_ERR_NULL;
    if (!aligned(m, 16) || !aligned(v, 16)) return ZS_ERR_UNSUPPORTED;
    const Range states[] = {span(m, state_elements * 4), span(v, state_elements * 4)};
    if (aliased(states, 2, nullptr, 0) || meets_state(tensors, n_tensors, states, 2))
        return ZS_ERR_ALIAS;
    return hip_status(zs::launch_adamw(tensors, n_tensors, constants(*config), m, v,
                                       static_cast<hipStream_t>(stream)));
}

int zs_adamw_step8(const zs_adamw_tensor* tensors, int64_t n_tensors,
                   const zs_adamw_config* config, uint8_t* m_code, float* m_scale, uint8_t* v_code,
                   float* v_scale, int64_t state_elements, uint32_t seed, void* stream) {
    const int st = adamw_tensors(tensors, n_tensors, config, state_elements);
    if (st != ZS_OK) return st;
    if (state_elements % ZS_ADAMW_BLOCK != 0) return ZS_ERR_SHAPE;
    if (state_elements == 0 || n_tensors == 0) return ZS_OK;
    if (!m_code || !m_scale || !v_code || !v_scale) return ZS_ERR_NULL;
    if (!aligned(m_code, 4) || !aligned(v_code, 4) || !aligned(m_scale, 4) || !aligned(v_scale, 4))
        return ZS_ERR_UNSUPPORTED;
    const int64_t blocks = state_elements / ZS_ADAMW_BLOCK;
    const Range states[] = {span(m_code, state_elements), span(v_code, state_elements),
                            span(m_scale, blocks * 4), span(v_scale, blocks * 4)};
    if (aliased(states, 4, nullptr, 0) || meets_state(tensors, n_tensors, states, 4))
        return ZS_ERR_ALIAS;
    return hip_status(zs::launch_adamw8(tensors, n_tensors, constants(*config), m_code, m_scale,
                                        v_code, v_scale, seed + uint32_t(config->step),
                                        static_cast<hipStream_t>(stream)));
}

int zs_adamw_moments8(const uint8_t* m_code, const float* m_scale, const uint8_t* v_code,
                      const float* v_scale, int64_t state_elements, float* m, float* v,
                      void* stream) {
    if (state_elements < 0 || state_elements > kMaxExtent / 8 ||
        state_elements % ZS_ADAMW_BLOCK != 0)
        return ZS_ERR_SHAPE;
    if (state_elements == 0) return ZS_OK;
    if (!m_code || !m_scale || !v_code || !v_scale || !m || !v) return ZS_ERR_NULL;
    if (!aligned(m_code, 4) || !aligned(v_code, 4) || !aligned(m_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(m, 16) || !aligned(v, 16))
        return ZS_ERR_UNSUPPORTED;
    const int64_t blocks = state_elements / ZS_ADAMW_BLOCK;
    const Range outs[] = {span(m, state_elements * 4), span(v, state_elements * 4)};
    const Range ins[] = {span(m_code, state_elements), span(v_code, state_elements),
                         span(m_scale, blocks * 4), span(v_scale, blocks * 4)};
    if (aliased(outs, 2, ins, 4)) return ZS_ERR_ALIAS;
    return hip_status(zs::launch_moments8(m_code, m_scale, v_code, v_scale, state_elements, m, v,
                                          static_cast<hipStream_t>(stream)));
}

}  // extern "C"
