"""Float64 references of the lookup, the layer norm, the router and the weighted sum, with the error bounds the tests
hold the kernels to (plain torch on the CPU, no code shared with the library)."""
import math

import torch

from blockref import ULP, sum_bound

HALF = 2.0 ** -24   # half an fp32 ulp, relative


def rounded(ref, inner, dtype):
    """A value within `inner` of ref, rounded once to the output type."""
    return inner + ULP[dtype] * (ref.abs() + inner) + 1e-38


# ---- lookup -----------------------------------------------------------------------------------------------------

def embedding(table, index, scale):
    """(y, bound): one fp32 product, rounded."""
    table = table.double()
    V = table.shape[0]
    live = (index >= 0) & (index < V)
    y = torch.where(live[:, None], table[index.clamp(0, V - 1)] * scale, 0.0)
    return y, lambda dtype: rounded(y, 2 * HALF * y.abs(), dtype)   # the scale is rounded to fp32 too


def embedding_grad(gy, index, V, scale):
    gy = gy.double()
    live = (index >= 0) & (index < V)
    out = torch.zeros(V, gy.shape[1], dtype=torch.float64).index_add_(0, index[live], gy[live])
    size = torch.zeros_like(out).index_add_(0, index[live], gy[live].abs())
    terms = int(torch.bincount(index[live], minlength=1).max()) if live.any() else 0
    return out * scale, lambda dtype: sum_bound(out * scale, size * abs(scale), terms + 2, dtype)


# ---- layer norm -------------------------------------------------------------------------------------------------

def norm_parts(x, eps):
    x = x.double()
    d = x - x.mean(1, keepdim=True)
    r = (d.square().mean(1, keepdim=True) + eps) ** -0.5
    return d * r, r


def layer_norm(x, w, b, eps):
    """(y, bound).  A row's sums take at most 48 additions one behind the other (32 values of a lane, six steps
    across a wavefront, eight wavefronts), each off by half an ulp of a partial sum of magnitudes: the mean is off by
    48 half ulps of the mean |d|, the factor r by half of that, and a handful of products follow."""
    xh, _ = norm_parts(x, eps)
    y = xh * w.double() + (0 if b is None else b.double())
    inner = HALF * (64 * (xh.abs() + 1) * w.double().abs() + (0 if b is None else 4 * b.double().abs()))
    return y, lambda dtype: rounded(y, inner, dtype)


def layer_norm_grads(gy, x, w, eps):
    """((gx, gw, gb), bounds): the sums as above, with xh off by 64 half ulps of |xh| + 1."""
    xh, r = norm_parts(x, eps)
    gy, w = gy.double(), w.double()
    t = gy * w
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    gx = r * (t - mean(t) - xh * mean(t * xh))
    inner = 128 * HALF * r * (t.abs() + mean(t.abs()) + (xh.abs() + 1) * (mean((t * xh).abs()) + mean(t.abs())))
    gw, gb = (gy * xh).sum(0), gy.sum(0)
    n = x.shape[0]
    bw = lambda: sum_bound(gw, (gy * xh).abs().sum(0), n, torch.float32) + 64 * HALF * (gy.abs() * (xh.abs() + 1)).sum(0)  # noqa: E731
    return (gx, gw, gb), (lambda dtype: rounded(gx, inner, dtype), bw, lambda: sum_bound(gb, gy.abs().sum(0), n, torch.float32))


# ---- routing ----------------------------------------------------------------------------------------------------

def scores(x, sigmoid):
    x = x.double()
    if sigmoid:
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    s = p.sum(1, keepdim=True)
    return p / torch.where(s == 0, 1.0, s)


def route(x, r, bias):
    """(weight, expert) in float64 and int64, row by row from the definition."""
    x = x.double()
    M, E = x.shape
    sigmoid, per = r.score == "sigmoid", E // r.groups
    s = scores(x, sigmoid)
    bad = x.isnan().any(1) | ((x == math.inf).any(1) if not sigmoid else torch.zeros(M, dtype=torch.bool))
    weight, expert = torch.zeros(M, r.k, dtype=torch.float64), torch.full((M, r.k), E)
    for t in range(M):
        if bad[t]:
            weight[t] = math.nan
            continue
        there = [e for e in range(E) if x[t, e] > -math.inf and (bias is None or bias[e] > -math.inf)]
        q = {e: float(s[t, e]) + (0.0 if bias is None else float(bias[e])) for e in there}
        if r.groups > 1:
            group = {}
            for e in there:
                group.setdefault(e // per, []).append(q[e])
            score = {g: sum(sorted(v, reverse=True)[:r.best]) for g, v in group.items()}
            stay = sorted(score, key=lambda g: (-score[g], g))[:r.top_groups]
            there = [e for e in there if e // per in stay]
        rank = q if bias is not None else {e: float(x[t, e]) for e in there}
        chosen = sorted(there, key=lambda e: (-rank[e], e))[:r.k]
        for j, e in enumerate(chosen):
            expert[t, j] = e
    w = shares(x, expert, r)[0 if r.renormalise else 1]
    return torch.where(bad[:, None], weight, r.scale * w), expert


def shares(x, expert, r):
    """(p, s) of the slots: shares of their sum, and scores; 0 where no expert is."""
    E = x.shape[1]
    live = (expert >= 0) & (expert < E)
    at = torch.where(live, expert, 0)
    sc = torch.where(live, scores(x, r.score == "sigmoid").gather(1, at), 0.0)
    p = sc
    if r.score == "softmax":
        v = torch.where(live, x.double().gather(1, at), -math.inf)
        top = v.amax(1, keepdim=True)
        p = torch.where(live, torch.exp(v - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = p.sum(1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), sc


def route_grad(gw, x, expert, r):
    """(gx, bound): the slots' parts are formed in 64 bits, a difference of terms of size p |g| and p sum |g| p whose
    roundings are 2^-53 each (up to 64 additions and a handful of products); a softmax's part of
    every logit is a product of two rounded factors, and the two parts are added in fp32.  The softmax's exponentials are
    fp32: one is off by an ulp and by |d| half ulps for the rounding of its argument d = x - max, and their sum by as
    much on average (|d| < 7 there, see the router's test)."""
    x = x.double()
    E = x.shape[1]
    live = (expert >= 0) & (expert < E)
    p, s = shares(x, expert, r)
    g = torch.where(live, gw.double() * r.scale, 0.0)
    if r.renormalise:
        d = p * (g - (g * p).sum(1, keepdim=True))
        if r.score == "sigmoid":
            d = d * (1 - s)
    else:
        d = g * s * (1 - s) if r.score == "sigmoid" else g * s
    out = torch.zeros(x.shape[0], E + 1, dtype=torch.float64).scatter_add_(1, torch.where(live, expert, E), d)[:, :E]
    terms = p * (g.abs() + (g * p).abs().sum(1, keepdim=True)) if r.renormalise else d.abs()
    wide = 128 * 2.0 ** -53 * torch.zeros(x.shape[0], E + 1, dtype=torch.float64).scatter_add_(1, torch.where(live, expert, E), terms)[:, :E]
    size = torch.zeros_like(out)
    if r.score == "softmax" and not r.renormalise:
        part = torch.where(live.any(1, keepdim=True), scores(x, False) * (g * s).sum(1, keepdim=True), 0.0)
        d = x - x.amax(1, keepdim=True)
        part_size = part.abs() * (8 + 7 + torch.where(d > -200, d.abs(), 0.0)) / 8   # below -200 the part is 0
        out, size = out - part, part_size + 15 / 8 * out.abs()
    return out, lambda dtype: rounded(out, HALF * (8 * size + 4 * out.abs()) + wide, dtype)


# ---- weighted sum -----------------------------------------------------------------------------------------------

def combine(z, weight):
    M, k = weight.shape
    t = z.double().reshape(M, k, z.shape[1]) * weight.double()[:, :, None]
    y = t.sum(1)
    return y, lambda dtype: sum_bound(y, t.abs().sum(1), k, dtype)


def combine_grads(gy, z, weight):
    M, k = weight.shape
    gz = (weight.double()[:, :, None] * gy.double()[:, None]).reshape(M * k, z.shape[1])
    t = gy.double()[:, None] * z.double().reshape(M, k, z.shape[1])
    gw = t.sum(2)
    return (gz, gw), (lambda dtype: rounded(gz, HALF * gz.abs(), dtype),
                      lambda: sum_bound(gw, t.abs().sum(2), z.shape[1], torch.float32))
