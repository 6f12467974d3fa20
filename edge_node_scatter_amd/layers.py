"""Binding of the operators before, between and behind the products of a block of experts (C ABI in
``include/zs_layers.h``):

* ``zs_embedding(table, index, scale)`` -> y, ``zs_embedding_backward(grad_y, index, n_entries, scale, groups)``, and
  the autograd function ``embedding``: rows looked up by token or species; the gradient sums them in sorted order.
* ``zs_layer_norm(x, w, b, eps)`` -> y, ``zs_layer_norm_backward``, and the autograd function ``layer_norm``.
* ``Router(n_experts, k, ...)``, ``zs_route(logits, router, bias)`` -> (weight, expert), ``zs_route_backward``, the
  autograd function ``route``, and ``expert_groups(expert, n_experts)``, the groups that ``grouped_mm`` reads.
* ``zs_combine(z, weight)`` -> y, ``zs_combine_backward``, and the autograd function ``combine``: the weighted sum of
  the experts' rows of a token.

As in the rest of the package these functions only marshal arguments; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os

import torch

from . import HEADER_PATH, Csr, _call, _check, _ptr, load, zs_build_csr
from .block import DTYPES, _check_groups, _rows, _typed

LAYERS_HEADER_PATH = os.path.join(os.path.dirname(HEADER_PATH), "zs_layers.h")
MAX_LAYER_WIDTH, MAX_EXPERTS, MAX_SLOTS, MAX_EXPERT_GROUPS = 8192, 1024, 64, 64

_layers_lib = None


class _Router(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("sigmoid", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("best", ctypes.c_int32),
                ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


def load_layers() -> ctypes.CDLL:
    """libzs.so with the signatures of include/zs_layers.h."""
    global _layers_lib
    if _layers_lib is None:
        lib = load()
        P, I64, SZ, INT, F32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int,
                                ctypes.c_float)
        R = ctypes.POINTER(_Router)
        sigs = {
            "zs_embedding": ([P, I64, P, I64, I64, I64, F32, INT, P, P], INT),
            "zs_embedding_backward_workspace_bytes": ([I64, I64, INT], SZ),
            "zs_embedding_backward": ([P, I64, P, P, P, I64, I64, I64, F32, INT, P, P, SZ, P], INT),
            "zs_layer_norm": ([P, I64, P, P, I64, I64, F32, INT, P, P], INT),
            "zs_layer_norm_workspace_bytes": ([I64, I64], SZ),
            "zs_layer_norm_backward": ([P, I64, P, I64, P, I64, I64, F32, INT, P, P, P, P, SZ, P],
                                       INT),
            "zs_route": ([P, I64, P, R, I64, I64, INT, P, P, P], INT),
            "zs_route_backward": ([P, P, I64, P, R, I64, I64, INT, P, P], INT),
            "zs_combine": ([P, I64, P, I64, I64, I64, INT, P, P], INT),
            "zs_combine_backward": ([P, I64, P, I64, P, I64, I64, I64, INT, P, P, P], INT),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _layers_lib = lib
    return _layers_lib


def _matrix(t: torch.Tensor, name: str, dtype: torch.dtype | None = None,
            device: torch.device | None = None):
    """A checked matrix with contiguous rows, its shape and its row stride (a single
    row's says nothing)."""
    if _typed(t, name, dtype, device).dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if t.is_contiguous():   # the usual case
        M, c = t.shape
        return t, M, c, c
    t = _rows(t)
    M, c = t.shape
    return t, M, c, t.stride(0) if M > 1 else c


def _dense(t: torch.Tensor, name: str, shape: tuple, dtype: torch.dtype,
           device: torch.device) -> torch.Tensor:
    """A checked tensor of one shape, contiguous."""
    if _typed(t, name, dtype, device).shape != shape:   # (a torch.Size is a tuple)
        raise ValueError(f"{name} must be {shape}")
    return t if t.is_contiguous() else t.contiguous()


def _workspace(size: int, device: torch.device) -> torch.Tensor | None:
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


# ---- lookup ----------------------------------------------------------------------------------------

def _index(index: torch.Tensor, device: torch.device) -> torch.Tensor:
    if _typed(index, "index", torch.int64, device).dim() != 1:
        raise ValueError("index must be (M,)")
    return index if index.is_contiguous() else index.contiguous()


def zs_embedding(table: torch.Tensor, index: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """y (M, c) with y[i] = scale * table[index[i]]; table (V, c) float32 or
    bfloat16, index (M,) int64.  The table may have a row stride.  Indices
    outside [0, V) (padding) give zeros."""
    table, V, c, stride = _matrix(table, "table")
    dev = table.device
    index = _index(index, dev)
    M = index.shape[0]
    y = table.new_empty((M, c))
    _check("zs_embedding", _call(
        dev, load_layers().zs_embedding, table.data_ptr(), stride, index.data_ptr(), M, V, c, scale,
        DTYPES[table.dtype], y.data_ptr()))
    return y


def zs_embedding_backward(grad_y: torch.Tensor, index: torch.Tensor, n_entries: int,
                          scale: float = 1.0, groups: Csr | None = None) -> torch.Tensor:
    """grad_table (n_entries, c) of zs_embedding, of grad_y's type: the rows of
    each entry added in fp32, zeros for entries without any.  The order of the
    additions is fixed by the sizes and groups (the same bits from run to run),
    but goes by stretches of rows whose sums are joined, not row by row.

    The sorted order is ``groups``: the ``Csr`` of ``zs_build_csr(index,
    n_entries)`` or, for rows that already are in the order of their entries,
    ``sorted_groups(offsets)``; without it the CSR is built here, without a
    synchronisation."""
    grad_y, M, c, stride = _matrix(grad_y, "grad_y")
    dev = grad_y.device
    index = _index(index, dev)
    if index.shape[0] != M:
        raise ValueError(f"index must be ({M},)")
    if n_entries < 1:
        raise ValueError("n_entries must be positive")
    out = grad_y.new_empty((n_entries, c))
    lib, dtype = load_layers(), DTYPES[grad_y.dtype]
    size = lib.zs_embedding_backward_workspace_bytes(M, c, dtype)
    if groups is None:
        # row offsets, order, entries, flag and workspaces in one allocation.  The flag says
        # that there is padding, which is allowed: nobody looks at it.
        need = int(lib.zs_csr_workspace_bytes(M, n_entries))
        at, parts = 0, []
        for part in (4 * (n_entries + 1), 4 * M, 4 * M, 4, need, size):
            parts.append(at)
            at += -(-part // 256) * 256
        keep = torch.empty(at, dtype=torch.uint8, device=dev)
        rowptr, perm, entries, flag, csr_ws, ws = (keep.data_ptr() + p for p in parts)
        _check("zs_build_csr", _call(dev, lib.zs_build_csr, _ptr(index), M, n_entries, rowptr, perm,
                                     entries, None, csr_ws, need, flag))
    else:
        if groups.n_nodes != n_entries:
            raise ValueError(f"groups must be of {n_entries} entries")
        _check_groups(groups, M, dev)
        keep = _workspace(size, dev)
        rowptr, perm, ws = _ptr(groups.rowptr), _ptr(groups.perm), _ptr(keep)
    _check("zs_embedding_backward", _call(
        dev, lib.zs_embedding_backward, _ptr(grad_y), stride, _ptr(index), rowptr, perm, M,
        n_entries, c, scale, dtype, _ptr(out), ws, size))
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, index, scale, rowptr, perm):
        ctx.save_for_backward(index, rowptr, perm)
        ctx.scale, ctx.n_entries = scale, table.shape[0]
        return zs_embedding(table, index, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        index, rowptr, perm = ctx.saved_tensors
        groups = None if rowptr is None else Csr(rowptr, perm, None, ctx.n_entries)
        return zs_embedding_backward(grad_y, index, ctx.n_entries, ctx.scale, groups), *(None,) * 4


def embedding(table: torch.Tensor, index: torch.Tensor, scale: float = 1.0,
              groups: Csr | None = None) -> torch.Tensor:
    """Differentiable zs_embedding (no double backward); ``groups`` as in
    zs_embedding_backward, where the caller has them already."""
    if groups is not None and groups.n_nodes != table.shape[0]:
        raise ValueError(f"groups must be of {table.shape[0]} entries")
    return _Embedding.apply(table, index, scale, groups and groups.rowptr, groups and groups.perm)


# ---- layer norm --------------------------------------------------------------------------------------

def zs_layer_norm(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None,
                  eps: float = 1e-5) -> torch.Tensor:
    """y = (x - mean) / sqrt(variance + eps) * w + b over the last of (M, c).
    x is float32 or bfloat16 and may have a row stride; w and b are float32 (c,)."""
    x, M, c, stride = _matrix(x, "x")
    dev = x.device
    w = _dense(w, "w", (c,), torch.float32, dev)
    b = b if b is None else _dense(b, "b", (c,), torch.float32, dev)
    y = x.new_empty((M, c))
    _check("zs_layer_norm", _call(
        dev, load_layers().zs_layer_norm, x.data_ptr(), stride, w.data_ptr(), _ptr(b), M, c, eps,
        DTYPES[x.dtype], y.data_ptr()))
    return y


def zs_layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                           need_b: bool = True, eps: float = 1e-5):
    """(grad_x, grad_w, grad_b) of zs_layer_norm; grad_b is None unless ``need_b``."""
    x, M, c, stride = _matrix(x, "x")
    dev = x.device
    grad_y, gM, gc, g_stride = _matrix(grad_y, "grad_y", x.dtype, dev)
    if (gM, gc) != (M, c):
        raise ValueError("grad_y must have x's shape")
    w = _dense(w, "w", (c,), torch.float32, dev)
    gx, gw = x.new_empty((M, c)), w.new_empty(c)
    gb = w.new_empty(c) if need_b else None
    lib = load_layers()
    size = lib.zs_layer_norm_workspace_bytes(M, c)
    ws = _workspace(size, dev)
    _check("zs_layer_norm_backward", _call(
        dev, lib.zs_layer_norm_backward, grad_y.data_ptr(), g_stride, x.data_ptr(), stride,
        w.data_ptr(), M, c, eps, DTYPES[x.dtype], gx.data_ptr(), gw.data_ptr(), _ptr(gb), _ptr(ws),
        size))
    return gx, gw, gb


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, eps):
        ctx.save_for_backward(x, w)
        ctx.has_b, ctx.eps = b is not None, eps
        return zs_layer_norm(x, w, b, eps)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        x, w = ctx.saved_tensors
        return (*zs_layer_norm_backward(grad_y, x, w, ctx.has_b, ctx.eps), None)


def layer_norm(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Differentiable zs_layer_norm (no double backward)."""
    return _LayerNorm.apply(x, w, b, eps)


# ---- routing -----------------------------------------------------------------------------------------

@dataclasses.dataclass(frozen=True)
class Router:
    """How rows choose their experts (include/zs_layers.h has the definition).

    ``score``: "softmax" or "sigmoid" of the logits.  ``groups``: the experts
    in that many groups of consecutive ones, of which the ``top_groups`` stay
    whose ``best`` (1 or 2) largest scores have the largest sum.  ``k``
    experts are chosen from those; their scores are the weights, divided by
    their sum if ``renormalise``, times ``scale``."""
    n_experts: int
    k: int
    score: str = "softmax"
    groups: int = 1
    top_groups: int = 1
    best: int = 2
    renormalise: bool = True
    scale: float = 1.0

    def __post_init__(self):
        if self.score not in ("softmax", "sigmoid"):
            raise ValueError("score must be 'softmax' or 'sigmoid'")
        if not 1 <= self.n_experts <= MAX_EXPERTS:
            raise ValueError(f"n_experts must be 1 to {MAX_EXPERTS}")
        if not 1 <= self.groups <= MAX_EXPERT_GROUPS or self.n_experts % self.groups:
            raise ValueError(f"groups must be 1 to {MAX_EXPERT_GROUPS} and divide n_experts")
        if not 1 <= self.top_groups <= self.groups:
            raise ValueError("top_groups must be 1 to groups")
        if not 1 <= self.k <= min(MAX_SLOTS, self.n_experts // self.groups * self.top_groups):
            raise ValueError(f"k must be 1 to {MAX_SLOTS} and at most the experts that stay")
        if self.best not in (1, 2):
            raise ValueError("best must be 1 or 2")
        if not math.isfinite(self.scale):
            raise ValueError("scale must be finite")
        # the library's form of it, made once: a router does not change
        object.__setattr__(self, "_c", _Router(
            self.k, self.score == "sigmoid", self.groups, self.top_groups, self.best,
            bool(self.renormalise), self.scale))


def _logits(logits: torch.Tensor, router: Router):
    logits, M, E, stride = _matrix(logits, "logits")
    if E != router.n_experts:
        raise ValueError(f"logits must be (M, {router.n_experts})")
    return logits, M, E, stride


def zs_route(logits: torch.Tensor, router: Router, bias: torch.Tensor | None = None):
    """(weight (M, k) float32, expert (M, k) int64) of logits (M, E), float32 or
    bfloat16, with an optional bias (E,) float32 that has a part in the choice
    only.  Experts with a logit or bias of -inf, or a NaN bias, are not there; a
    slot that no expert is left for holds E and weight 0.  A row's results do not
    depend on the other rows of the call."""
    logits, M, E, stride = _logits(logits, router)
    dev = logits.device
    bias = bias if bias is None else _dense(bias, "bias", (E,), torch.float32, dev)
    weight = logits.new_empty((M, router.k), dtype=torch.float32)
    expert = logits.new_empty((M, router.k), dtype=torch.int64)
    _check("zs_route", _call(
        dev, load_layers().zs_route, logits.data_ptr(), stride, _ptr(bias), router._c, M, E,
        DTYPES[logits.dtype], weight.data_ptr(), expert.data_ptr()))
    return weight, expert


def zs_route_backward(grad_weight: torch.Tensor, logits: torch.Tensor, expert: torch.Tensor,
                      router: Router) -> torch.Tensor:
    """grad_logits (M, E) of zs_route from grad_weight (M, k) float32, the choice
    ``expert`` held fixed."""
    logits, M, E, stride = _logits(logits, router)
    dev = logits.device
    grad_weight = _dense(grad_weight, "grad_weight", (M, router.k), torch.float32, dev)
    expert = _dense(expert, "expert", (M, router.k), torch.int64, dev)
    out = logits.new_empty((M, E))
    _check("zs_route_backward", _call(
        dev, load_layers().zs_route_backward, grad_weight.data_ptr(), logits.data_ptr(), stride,
        expert.data_ptr(), router._c, M, E, DTYPES[logits.dtype], out.data_ptr()))
    return out


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, router):
        weight, expert = zs_route(logits, router, bias)
        ctx.save_for_backward(logits, expert)
        ctx.router = router
        ctx.mark_non_differentiable(expert)
        return weight, expert

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_weight, _):
        logits, expert = ctx.saved_tensors
        return zs_route_backward(grad_weight, logits, expert, ctx.router), None, None


def route(logits: torch.Tensor, router: Router, bias: torch.Tensor | None = None):
    """Differentiable zs_route (no double backward): the weights carry gradients
    to the logits, the choice and the bias carry none."""
    return _Route.apply(logits, bias, router)


def expert_groups(expert: torch.Tensor, n_experts: int) -> Csr:
    """The groups of the (M, k) experts that zs_route chose, for grouped_mm: row
    t * k + j belongs to expert[t, j].  Slots without an expert (index
    ``n_experts``) are rows of no group, whose products are zeros.  Indices
    outside [0, n_experts] are not looked for, as the groups are built without a
    synchronisation: products of such rows, and of others, are unspecified."""
    if _typed(expert, "expert", torch.int64).dim() != 2:
        raise ValueError("expert must be (M, k)")
    bad = torch.empty(1, dtype=torch.int32, device=expert.device)
    csr = zs_build_csr(expert.reshape(-1), n_experts + 1, bad_flag=bad, order=False)
    return Csr(csr.rowptr[:-1], csr.perm, csr.dst32, n_experts)


# ---- weighted sum --------------------------------------------------------------------------------------

def _slots(z: torch.Tensor, weight: torch.Tensor):
    """z, its width and row stride, weight and its shape, checked."""
    z, rows, c, stride = _matrix(z, "z")
    if _typed(weight, "weight", torch.float32, z.device).dim() != 2:
        raise ValueError("weight must be (M, k)")
    M, k = weight.shape
    if rows != M * k:
        raise ValueError("z must have a row for each of weight's entries")
    return z, c, stride, weight if weight.is_contiguous() else weight.contiguous(), M, k


def zs_combine(z: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """y (M, c) with y[t] = sum over j of weight[t, j] * z[t * k + j]; z (M * k, c)
    float32 or bfloat16, which may have a row stride, weight (M, k) float32."""
    z, c, stride, weight, M, k = _slots(z, weight)
    y = z.new_empty((M, c))
    _check("zs_combine", _call(
        z.device, load_layers().zs_combine, z.data_ptr(), stride, weight.data_ptr(), M, k, c,
        DTYPES[z.dtype], y.data_ptr()))
    return y


def zs_combine_backward(grad_y: torch.Tensor, z: torch.Tensor, weight: torch.Tensor):
    """(grad_z (M * k, c), grad_weight (M, k) float32) of zs_combine."""
    z, c, stride, weight, M, k = _slots(z, weight)
    grad_y, gM, gc, g_stride = _matrix(grad_y, "grad_y", z.dtype, z.device)
    if (gM, gc) != (M, c):
        raise ValueError(f"grad_y must be ({M}, {c})")
    gz, gw = z.new_empty((M * k, c)), weight.new_empty((M, k))
    _check("zs_combine_backward", _call(
        z.device, load_layers().zs_combine_backward, grad_y.data_ptr(), g_stride, z.data_ptr(),
        stride, weight.data_ptr(), M, k, c, DTYPES[z.dtype], gz.data_ptr(), gw.data_ptr()))
    return gz, gw


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, weight):
        ctx.save_for_backward(z, weight)
        return zs_combine(z, weight)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        return zs_combine_backward(grad_y, *ctx.saved_tensors)


def combine(z: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """Differentiable zs_combine (no double backward)."""
    return _Combine.apply(z, weight)
