"""Binding of the learned operators around the scatter (C ABI in ``include/zs_block.h``).

* ``zs_grouped_mm(x, w, groups)`` -> y, ``zs_grouped_mm_backward(grad_y, x, w, groups)`` -> (grad_x, grad_w),
  and the autograd function ``grouped_mm(x, w, groups)``: matrix products whose rows are grouped by species or
  expert.  ``groups`` is the ``Csr`` of ``zs_build_csr(index, n_groups)`` over the rows' group indices, or
  ``sorted_groups(offsets)`` for rows that already are in group order.
* ``zs_block_join(x, z, gate, scale, w_post, w_pre, eps)`` -> (y, h), ``zs_block_join_backward``, and the
  autograd functions ``block_join`` and ``block_norm``: the join of a block's output with its residual stream,
  from the norm behind the block to the norm before the next one.
* ``AdamW``: the optimizer step over all parameter tensors, with moments in 32 or 8 bits.

As in the rest of the package these functions only marshal arguments; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch
from torch.autograd.graph import increment_version

from . import HEADER_PATH, Csr, ZsError, _call, _check, _ptr, load

BLOCK_HEADER_PATH = os.path.join(os.path.dirname(HEADER_PATH), "zs_block.h")
STATE_BLOCK = 256
MAX_GROUPS, MAX_WIDTH, MAX_JOIN_WIDTH = 1 << 20, 65536, 8192
DTYPES = {torch.float32: 0, torch.bfloat16: 1}

_block_lib = None


class _Tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("state_offset", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _Config(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64)]


def load_block() -> ctypes.CDLL:
    """libzs.so with the signatures of include/zs_block.h."""
    global _block_lib
    if _block_lib is None:
        lib = load()
        P, I64, SZ, INT, F32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int,
                                ctypes.c_float)
        T, C = ctypes.POINTER(_Tensor), ctypes.POINTER(_Config)
        sigs = {
            "zs_grouped_mm": ([P, I64, P, I64, I64, INT, P, P, I64, I64, I64, I64, INT, P, I64, P],
                              INT),
            "zs_grouped_mm_wgrad_workspace_bytes": ([I64, I64, I64, I64, INT], SZ),
            "zs_grouped_mm_wgrad": ([P, I64, P, I64, P, P, I64, I64, I64, I64, INT, P, P, SZ, P],
                                    INT),
            "zs_grouped_mm_backward": ([P, I64, P, I64, P, I64, I64, P, P, I64, I64, I64, I64, INT,
                                        P, P, P, SZ, P], INT),
            "zs_block_join": ([P, I64, P, I64, P, I64, I64, P, P, P, I64, I64, F32, INT, P, P, P],
                              INT),
            "zs_block_join_workspace_bytes": ([I64, I64], SZ),
            "zs_block_join_backward": ([P, P, P, I64, P, I64, P, I64, I64, P, P, P, I64, I64, F32,
                                        INT, P, P, P, P, P, P, P, SZ, P], INT),
            "zs_adamw_step": ([T, I64, C, P, P, I64, P], INT),
            "zs_adamw_step8": ([T, I64, C, P, P, P, P, I64, ctypes.c_uint32, P], INT),
            "zs_adamw_moments8": ([P, P, P, P, I64, P, P, P], INT),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _block_lib = lib
    return _block_lib


def _typed(t: torch.Tensor, name: str, dtype: torch.dtype | None = None,
           device: torch.device | None = None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dtype is None:
        if t.dtype not in DTYPES:
            raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t


def _rows(t: torch.Tensor) -> torch.Tensor:
    """A matrix whose rows are contiguous: a view with a row stride is taken in
    place, anything else is copied."""
    row, col = t.stride()
    if (col != 1 and t.shape[1] > 1) or row < 0:
        t = t.contiguous()
    return t


# ---- grouped products ----------------------------------------------------------------------------

def sorted_groups(offsets: torch.Tensor) -> Csr:
    """Groups of rows that already are in group order: group g holds the rows
    offsets[g] .. offsets[g + 1] - 1 (int32, on the GPU)."""
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be (G + 1,)")
    return Csr(_typed(offsets, "offsets", torch.int32).contiguous(), None, None,
               offsets.numel() - 1)


def _check_groups(groups: Csr, n_rows: int, device: torch.device) -> None:
    _typed(groups.rowptr, "groups.rowptr", torch.int32, device)
    if tuple(groups.rowptr.shape) != (groups.n_nodes + 1,) or not groups.rowptr.is_contiguous():
        raise ValueError(f"groups.rowptr must be contiguous ({groups.n_nodes + 1},)")
    if groups.perm is not None:
        _typed(groups.perm, "groups.perm", torch.int32, device)
        if tuple(groups.perm.shape) != (n_rows,) or not groups.perm.is_contiguous():
            raise ValueError(f"groups.perm must be contiguous ({n_rows},)")


def _weights(w: torch.Tensor) -> tuple[torch.Tensor, int]:
    """w (G, k, n) and whether its memory is [n][k] (a transposed view, as of
    weights kept output-major); other layouts are copied."""
    group, row, col = w.stride()
    if (col == 1 or w.shape[2] == 1) and group >= 0 and row >= 0:
        return w, 0
    if (row == 1 or w.shape[1] == 1) and group >= 0 and col >= 0:
        return w, 1
    return w.contiguous(), 0


def _mm(x, w, transposed, groups, k, n, out):
    """out = x op(w): w's own strides, its memory [k][n] or, transposed, [n][k]."""
    row = w.stride(2) if transposed else w.stride(1)
    return _call(x.device, load_block().zs_grouped_mm, _ptr(x), x.stride(0), _ptr(w), w.stride(0),
                 row, transposed, _ptr(groups.rowptr), _ptr(groups.perm), x.shape[0],
                 groups.n_nodes, k, n, DTYPES[x.dtype], _ptr(out),
                 out.stride(0) if x.shape[0] > 1 else n)   # a single row's stride says nothing


def _mm_inputs(x, w, groups):
    """x and w, checked against each other and the groups; x with contiguous rows."""
    dtype, dev, xs, ws = x.dtype, x.device, x.shape, w.shape
    offsets, perm = groups.rowptr, groups.perm
    if not (x.is_cuda and dtype in DTYPES and w.dtype == dtype and w.device == dev
            and len(xs) == 2 and len(ws) == 3 and ws[0] == groups.n_nodes and ws[1] == xs[1]
            and offsets.dtype == torch.int32 and offsets.device == dev
            and offsets.shape == (ws[0] + 1,) and offsets.is_contiguous()
            and (perm is None or perm.dtype == torch.int32 and perm.device == dev
                 and perm.shape == xs[:1] and perm.is_contiguous())):
        _typed(x, "x")
        _typed(w, "w", dtype, dev)
        if len(xs) != 2 or len(ws) != 3 or ws[0] != groups.n_nodes or ws[1] != xs[1]:
            raise ValueError("x must be (M, k) and w (G, k, n), G the number of groups")
        _check_groups(groups, xs[0], dev)
        raise ValueError("inputs do not fit a grouped product")
    return _rows(x), w


def zs_grouped_mm(x: torch.Tensor, w: torch.Tensor, groups: Csr,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """y (M, n) with y[i] = x[i] @ w[group of row i]; x (M, k) and w (G, k, n)
    float32 or bfloat16 (accumulated in fp32).  x may have a row stride, w may
    be a transposed view; ``out`` may have a row stride of at least n.  Rows of
    no group get zeros."""
    x, w = _mm_inputs(x, w, groups)
    M, n, given = x.shape[0], w.shape[2], out is not None
    if not given:
        out = x.new_empty((M, n))
    else:
        _typed(out, "out", x.dtype, x.device)
        if tuple(out.shape) != (M, n) or (n > 1 and out.stride(1) != 1):
            raise ValueError(f"out must be ({M}, {n}) with contiguous rows")
    w, transposed = _weights(w)
    _check("zs_grouped_mm", _mm(x, w, transposed, groups, x.shape[1], n, out))
    if given:
        increment_version(out)
    return out


def _wgrad_workspace(M, n_groups, k, n, x):
    size = load_block().zs_grouped_mm_wgrad_workspace_bytes(M, n_groups, k, n, DTYPES[x.dtype])
    return torch.empty(size, dtype=torch.uint8, device=x.device) if size else None, size


def zs_grouped_mm_backward(grad_y: torch.Tensor, x: torch.Tensor, w: torch.Tensor, groups: Csr,
                           need_x: bool = True, need_w: bool = True):
    """(grad_x (M, k), grad_w (G, k, n)) of zs_grouped_mm; None for one that is
    not needed.  grad_w has w's dtype; a transposed view w gives a grad_w of the
    same strides."""
    x, w = _mm_inputs(x, w, groups)
    M, k, n = x.shape[0], w.shape[1], w.shape[2]
    grad_y = _typed(grad_y, "grad_y", x.dtype, x.device)
    if tuple(grad_y.shape) != (M, n):
        raise ValueError(f"grad_y must be ({M}, {n})")
    grad_y = _rows(grad_y)
    w, transposed = _weights(w)
    gx = gw = None
    if need_x and need_w and not transposed:
        gx = torch.empty((M, k), dtype=x.dtype, device=x.device)
        gw = torch.empty((groups.n_nodes, k, n), dtype=x.dtype, device=x.device)
        ws, size = _wgrad_workspace(M, groups.n_nodes, k, n, x)
        _check("zs_grouped_mm_backward", _call(
            x.device, load_block().zs_grouped_mm_backward, _ptr(grad_y), grad_y.stride(0), _ptr(x),
            x.stride(0), _ptr(w), w.stride(0), w.stride(1), _ptr(groups.rowptr), _ptr(groups.perm),
            M, groups.n_nodes, k, n, DTYPES[x.dtype], _ptr(gx), _ptr(gw), _ptr(ws), size))
        return gx, gw
    if need_x:
        gx = torch.empty((M, k), dtype=x.dtype, device=x.device)
        # the memory [k][n] read as the [n][k] of the transposed product
        wt = w.transpose(1, 2)
        _check("zs_grouped_mm", _mm(grad_y, wt, 1 - transposed, groups, n, k, gx))
    if need_w:
        a, b = (grad_y, x) if transposed else (x, grad_y)
        gw = torch.empty((groups.n_nodes, a.shape[1], b.shape[1]), dtype=x.dtype, device=x.device)
        ws, size = _wgrad_workspace(M, groups.n_nodes, a.shape[1], b.shape[1], x)
        _check("zs_grouped_mm_wgrad", _call(
            x.device, load_block().zs_grouped_mm_wgrad, _ptr(a), a.stride(0), _ptr(b), b.stride(0),
            _ptr(groups.rowptr), _ptr(groups.perm), M, groups.n_nodes, a.shape[1], b.shape[1],
            DTYPES[x.dtype], _ptr(gw), _ptr(ws), size))
        if transposed:
            gw = gw.transpose(1, 2)
    return gx, gw


class _GroupedMm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, rowptr, perm, n_groups):
        ctx.save_for_backward(x, w, rowptr, perm)
        ctx.n_groups = n_groups
        return zs_grouped_mm(x, w, Csr(rowptr, perm, None, n_groups))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        x, w, rowptr, perm = ctx.saved_tensors
        gx, gw = zs_grouped_mm_backward(grad_y, x, w, Csr(rowptr, perm, None, ctx.n_groups),
                                        ctx.needs_input_grad[0], ctx.needs_input_grad[1])
        return gx, gw, None, None, None


def grouped_mm(x: torch.Tensor, w: torch.Tensor, groups: Csr) -> torch.Tensor:
    """Differentiable zs_grouped_mm (no double backward)."""
    return _GroupedMm.apply(x, w, groups.rowptr, groups.perm, groups.n_nodes)


# ---- residual join ---------------------------------------------------------------------------------

def _join_refusal(x, z, gate, scale, w_post, w_pre):
    """Raises for what is wrong with a join's inputs, one by one."""
    _typed(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be (M, c)")
    dev, c = x.device, x.shape[1]
    if z is None:
        if gate is not None or scale is not None or w_post is not None:
            raise ValueError("gate, scale and w_post need z")
        if w_pre is None:
            raise ValueError("z or w_pre must be given")
    else:
        _typed(z, "z", x.dtype, dev)
        if z.shape != x.shape:
            raise ValueError("z must have x's shape")
        if scale is None or w_post is None:
            raise ValueError("z needs scale and w_post")
        if gate is not None:
            _typed(gate, "gate", x.dtype, dev)
            if tuple(gate.shape) not in ((x.shape[0], c), (x.shape[0], 1)):
                raise ValueError("gate must be (M, c) or (M, 1)")
    for name, t in (("scale", scale), ("w_post", w_post), ("w_pre", w_pre)):
        if t is not None:
            _typed(t, name, torch.float32, dev)
            if tuple(t.shape) != (c,):
                raise ValueError(f"{name} must be ({c},)")


def _join_inputs(x, z, gate, scale, w_post, w_pre):
    """The inputs, checked, as the kernels can read them."""
    F32, dev, shape, dtype = torch.float32, x.device, x.shape, x.dtype
    ok = x.is_cuda and dtype in DTYPES and len(shape) == 2
    if ok:
        c = shape[1:]
        if z is None:
            ok = gate is None and scale is None and w_post is None and w_pre is not None
        else:
            ok = (scale is not None and w_post is not None and z.shape == shape
                  and z.dtype == dtype and z.device == dev
                  and scale.shape == c and scale.dtype == F32 and scale.device == dev
                  and w_post.shape == c and w_post.dtype == F32 and w_post.device == dev
                  and (gate is None or gate.dtype == dtype and gate.device == dev
                       and (gate.shape == shape or gate.shape == (shape[0], 1))))
        ok = ok and (w_pre is None or w_pre.shape == c and w_pre.dtype == F32
                     and w_pre.device == dev)
    if not ok:
        _join_refusal(x, z, gate, scale, w_post, w_pre)
        raise ValueError("inputs do not fit a join")
    return (_rows(x), z if z is None else _rows(z), gate if gate is None else _rows(gate),
            *(t if t is None or t.is_contiguous() else t.contiguous()
              for t in (scale, w_post, w_pre)))


def _join_args(x, z, gate, scale, w_post, w_pre, eps):
    # an empty tensor has no address; z's says whether there is a block at all
    z_ptr = None if z is None else z.data_ptr() or w_post.data_ptr()
    return (_ptr(x), x.stride(0), z_ptr, 0 if z is None else z.stride(0), _ptr(gate),
            0 if gate is None else gate.stride(0), 0 if gate is None else gate.shape[1],
            _ptr(scale), _ptr(w_post), _ptr(w_pre), x.shape[0], x.shape[1], eps, DTYPES[x.dtype])


def zs_block_join(x: torch.Tensor, z: torch.Tensor | None, gate: torch.Tensor | None,
                  scale: torch.Tensor | None, w_post: torch.Tensor | None,
                  w_pre: torch.Tensor | None, eps: float = 1e-6):
    """(y, h): y = x + scale * sigmoid(gate) * rmsnorm(z) * w_post and
    h = rmsnorm(y) * w_pre, norms over the last of (M, c).

    x, z and gate are float32 or bfloat16 and may have a row stride; gate is
    (M, c), (M, 1) or None; scale, w_post and w_pre are float32 (c,).  h is None
    when w_pre is; without z, y is x itself and h its norm."""
    given = x
    x, z, gate, scale, w_post, w_pre = _join_inputs(x, z, gate, scale, w_post, w_pre)
    y = given if z is None else x.new_empty(x.shape)
    h = None if w_pre is None else x.new_empty(x.shape)
    _check("zs_block_join", _call(
        x.device, load_block().zs_block_join, *_join_args(x, z, gate, scale, w_post, w_pre, eps),
        None if z is None else _ptr(y), _ptr(h)))
    return y, h


def zs_block_join_backward(grad_y: torch.Tensor | None, grad_h: torch.Tensor | None,
                           x: torch.Tensor, z: torch.Tensor | None, gate: torch.Tensor | None,
                           scale: torch.Tensor | None, w_post: torch.Tensor | None,
                           w_pre: torch.Tensor | None, eps: float = 1e-6):
    """(grad_x, grad_z, grad_gate, grad_scale, grad_w_post, grad_w_pre), None
    for inputs that are None.  grad_y or grad_h may be None (zeros)."""
    x, z, gate, scale, w_post, w_pre = _join_inputs(x, z, gate, scale, w_post, w_pre)
    dev, shape, (M, c) = x.device, x.shape, x.shape
    for name, g in (("grad_y", grad_y), ("grad_h", grad_h)):
        if g is not None and not (g.dtype == x.dtype and g.device == dev and g.shape == shape):
            _typed(g, name, x.dtype, dev)
            raise ValueError(f"{name} must have x's shape")
    grad_y = grad_y if grad_y is None or grad_y.is_contiguous() else grad_y.contiguous()
    grad_h = grad_h if grad_h is None or grad_h.is_contiguous() else grad_h.contiguous()
    gx = x.new_empty(shape)
    gz = None if z is None else x.new_empty(shape)
    gg = None if gate is None else x.new_empty(gate.shape)
    # the parameters' gradients in one allocation
    gs, gpost, gpre = torch.empty((3, c), dtype=torch.float32, device=dev).unbind(0)
    if z is None:
        gs = gpost = None
    if w_pre is None:
        gpre = None
    lib = load_block()
    size = lib.zs_block_join_workspace_bytes(M, c)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _check("zs_block_join_backward", _call(
        dev, lib.zs_block_join_backward, _ptr(grad_y), _ptr(grad_h),
        *_join_args(x, z, gate, scale, w_post, w_pre, eps), _ptr(gx), _ptr(gz), _ptr(gg),
        _ptr(gs), _ptr(gpost), _ptr(gpre), _ptr(ws), size))
    return gx, gz, gg, gs, gpost, gpre


class _BlockJoin(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, gate, scale, w_post, w_pre, eps):
        ctx.save_for_backward(x, z, gate, scale, w_post, w_pre)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        y, h = zs_block_join(x, z, gate, scale, w_post, w_pre, eps)
        return h if z is None else ((y, h) if h is not None else y)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        x, z, gate, scale, w_post, w_pre = ctx.saved_tensors
        if z is None:
            gy, gh = None, grads[0]
        else:
            gy, gh = grads[0], grads[1] if w_pre is not None else None
        if gy is None and gh is None:
            return (None,) * 7
        return (*zs_block_join_backward(gy, gh, x, z, gate, scale, w_post, w_pre, ctx.eps), None)


def block_join(x: torch.Tensor, z: torch.Tensor, gate: torch.Tensor | None, scale: torch.Tensor,
               w_post: torch.Tensor, w_pre: torch.Tensor | None = None, eps: float = 1e-6):
    """Differentiable zs_block_join (no double backward): (y, h), or y alone
    when w_pre is None."""
    return _BlockJoin.apply(x, z, gate, scale, w_post, w_pre, eps)


def block_norm(x: torch.Tensor, w_pre: torch.Tensor, eps: float = 1e-6) -> torch.Tensor:
    """Differentiable rmsnorm(x) * w_pre: the norm before the first block."""
    return _BlockJoin.apply(x, None, None, None, None, w_pre, eps)


# ---- AdamW -------------------------------------------------------------------------------------------

_dtype_of, _nbytes_of = torch.Tensor.dtype.__get__, torch.Tensor.nbytes.__get__


class AdamW:
    """AdamW over many fp32 parameter tensors, one kernel launch for up to 64
    of them.  Moments lie in one flat array each, tensor i from
    ``offsets[i]`` (a multiple of 256) on.

    ``state_bits`` 32: ``state["m"]`` and ``state["v"]`` fp32.  8: codes with a
    scale per 256 elements (``m_code``, ``m_scale``, ``v_code``, ``v_scale``,
    and the integer ``seed`` of the stochastic rounding); the format is in
    include/zs_block.h.  ``state["step"]`` counts the steps done.

    ``copies``: bf16 tensors that receive each new parameter rounded (the
    working copies that bf16 products read), or None.  ``state``: an earlier
    ``AdamW.state``, taken over in place.

    Rate and decay are one for all of an object's tensors: tensors that shall
    not decay take an object of their own.  A step captured in a HIP graph is
    counted once, at the capture, and every replay is that step again (the same
    bias corrections and random bits): capture what leads up to it instead.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, copies=None, seed: int = 0,
                 state: dict | None = None):
        self.params = list(params)
        if not self.params:
            raise ValueError("params is empty")
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        self.device = _typed(self.params[0], "params[0]", torch.float32).device
        self.copies = None if copies is None else list(copies)
        if self.copies is not None and len(self.copies) != len(self.params):
            raise ValueError("copies must be one tensor for each parameter")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits = state_bits
        self.offsets, total = [], 0
        for i, p in enumerate(self.params):
            self._dense(p, f"params[{i}]", torch.float32, p.shape)
            if self.copies is not None:
                self._dense(self.copies[i], f"copies[{i}]", torch.bfloat16, p.shape)
            self.offsets.append(total)
            total += -(-p.numel() // STATE_BLOCK) * STATE_BLOCK
        self.total = total
        names = {32: ("m", "v"), 8: ("m_code", "m_scale", "v_code", "v_scale")}[state_bits]
        if state is None:
            state = {"step": 0, **{n: torch.zeros(self._shape(n), dtype=self._dtype(n),
                                                  device=self.device) for n in names}}
            if state_bits == 8:
                state["seed"] = seed
        self._arrays = [(n, self._dtype(n), torch.Size(self._shape(n))) for n in names]
        self.state = dict(state)
        self._state()
        self._table = (_Tensor * len(self.params))()
        # the table as 64-bit words: param, grad, copy, n, state_offset, grad_dtype and reserved
        self._words = (ctypes.c_int64 * (6 * len(self.params))).from_buffer(self._table)
        self._shapes = [p.shape for p in self.params]
        self._words[3::6] = self._sizes = [p.numel() for p in self.params]
        self._bytes = [4 * n for n in self._sizes], [2 * n for n in self._sizes]
        self._words[4::6] = self.offsets
        self._missing = False   # whether the table's sizes have zeros for missing gradients
        self._apart(self._addresses())

    def _shape(self, name):
        return (self.total // STATE_BLOCK,) if name.endswith("_scale") else (self.total,)

    @staticmethod
    def _dtype(name):
        return torch.uint8 if name.endswith("_code") else torch.float32

    def _dense(self, t, name, dtype, shape):
        _typed(t, name, dtype, self.device)
        if t.shape != torch.Size(shape) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {tuple(shape)}")

    def step(self, grads=None) -> None:
        """One step with ``grads`` (fp32 or bf16, one for each parameter; None:
        the parameters' ``grad``).  A parameter whose gradient is None keeps
        its value and moments."""
        if grads is None:
            grads = [p.grad for p in self.params]
        if len(grads) != len(self.params):
            raise ValueError("grads must be one tensor for each parameter")
        self._fill(grads)
        s = self.state
        c = _Config(self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay,
                    s["step"] + 1)
        lib = load_block()
        at = self._state()
        if self.state_bits == 32:
            status = _call(self.device, lib.zs_adamw_step, self._table, len(self._table), c, *at,
                           self.total)
        else:
            status = _call(self.device, lib.zs_adamw_step8, self._table, len(self._table), c, *at,
                           self.total, s["seed"] & 0xFFFFFFFF)
        _check("zs_adamw_step", status)
        s["step"] += 1
        # what the kernel wrote counts as changed in place, for graphs that saved it
        written = self.params if self.copies is None else self.params + self.copies
        if self._missing:
            written = [t for t, g in zip(written, list(grads) * 2) if g is not None]
        increment_version(written)

    def _same(self, tensors, sizes) -> bool:
        """Whether tensors still have the bytes, device and layout that they had: a
        tensor's memory can be replaced behind the optimizer (``module.bfloat16()``
        keeps the Parameter and gives it another type's).  The type itself is looked
        at where an address changed."""
        T = torch.Tensor
        return (list(map(_nbytes_of, tensors)) == sizes
                and set(map(T.get_device, tensors)) == {self.device.index}
                and all(map(T.is_contiguous, tensors)))

    def _state(self) -> list[int]:
        """Addresses of the state arrays, in the calls' order, each looked at: the
        dictionary is the caller's to change."""
        at = []
        for name, dtype, shape in self._arrays:
            t = self.state[name]
            if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape
                    or t.get_device() != self.device.index or not t.is_contiguous()):
                self._dense(t, f"state[{name!r}]", dtype, shape)
            at.append(t.data_ptr())
        return at

    def _addresses(self) -> list[int]:
        """Of the parameters, then of the copies."""
        T = torch.Tensor
        at = list(map(T.data_ptr, self.params))
        return at if self.copies is None else at + list(map(T.data_ptr, self.copies))

    def _apart(self, at) -> None:
        """Parameters and copies at these addresses from here on, unless they share
        memory there: one launch writes them all, in no order."""
        n = len(self.params)
        ranges = sorted((a, a + (4 if i < n else 2) * self._sizes[i % n])
                        for i, a in enumerate(at) if self._sizes[i % n])
        if any(a[1] > b[0] for a, b in zip(ranges, ranges[1:])):
            raise ValueError("parameters and copies must not share memory")
        self._words[0::6] = at[:n]
        if self.copies is not None:
            self._words[2::6] = at[n:]
        self._at = at

    def _fill(self, grads) -> None:
        """The table's addresses and types for this step.  All tensors are looked
        at in a few passes over the lists; what a pass finds is named one by one."""
        T, words, params, sizes = torch.Tensor, self._words, self.params, self._sizes
        missing = type(None) in set(map(type, grads))
        if missing:
            # a tensor without a gradient gets a size of 0 and its own memory's address
            sizes = [0 if g is None else n for g, n in zip(grads, sizes)]
            grads = [p if g is None else g for g, p in zip(grads, params)]
        types = list(map(DTYPES.get, map(_dtype_of, grads)))
        at = self._addresses()
        if (None in types or at != self._at or [g.shape for g in grads] != self._shapes
                or set(map(T.get_device, grads)) != {self.device.index}
                or not all(map(T.is_contiguous, grads)) or not self._same(params, self._bytes[0])
                or self.copies is not None and not self._same(self.copies, self._bytes[1])):
            for i, (g, shape) in enumerate(zip(grads, self._shapes)):
                self._dense(params[i], f"params[{i}]", torch.float32, shape)
                if self.copies is not None:
                    self._dense(self.copies[i], f"copies[{i}]", torch.bfloat16, shape)
                if g.dtype not in DTYPES:
                    raise TypeError(f"grads[{i}] must be float32 or bfloat16, got {g.dtype}")
                self._dense(g, f"grads[{i}]", g.dtype, shape)
            self._apart(at)
        words[1::6] = list(map(T.data_ptr, grads))
        if missing or self._missing:
            words[3::6] = sizes
        self._missing = missing
        words[5::6] = types

    def moments(self) -> tuple[torch.Tensor, torch.Tensor]:
        """(m, v) flat in fp32: the state itself with 32 bits, the values that
        its codes stand for with 8."""
        if self.state_bits == 32:   # the caller's own arrays: nothing reads them here
            return self.state["m"], self.state["v"]
        at = self._state()
        m = torch.empty(self.total, dtype=torch.float32, device=self.device)
        v = torch.empty_like(m)
        _check("zs_adamw_moments8", _call(
            self.device, load_block().zs_adamw_moments8, *at, self.total, _ptr(m), _ptr(v)))
        return m, v
