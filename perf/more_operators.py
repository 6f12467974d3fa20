"""Measured cases of the operators before, between and behind the products of a block of experts: embedding lookup with
its gradient by sorted rows, layer norm, routing to experts, and the weighted sum of the experts' outputs.

``listed`` and ``draw`` give the cases, ``prepare`` makes a case's inputs on the GPU from a seed, ``run`` does one
pass: the plain form in elementary torch operations where ``own`` is false, the framework's kernels where it is
true.  ``exact`` is the same pass from the definitions in float64.

Definitions (rows i, widths c, experts e, slots j < k of a row):

  embedding  y[i] = a T[index[i]], 0 where index[i] is outside [0, V)
             dT[v] = a * sum over the rows i with index[i] = v of dy[i]
  norm       mu = mean x, r = (mean (x - mu)^2 + eps)^(-1/2), xh = (x - mu) r, y = xh w + b
             t = dy w, dx = r (t - mean t - xh mean(t xh)), dw = sum of dy xh, db = sum of dy over the rows
  route      s = softmax(x) or sigmoid(x) of a row, q = s + bias.  An expert whose logit or bias is -inf is not there.
             The groups of experts with the largest sums of their best (one or two) q stay, then the k experts of
             largest q (without bias: of largest x) of those; ties go to the lowest index.
             w_j = a s_ij, or a s_ij / sum_l s_il; a slot that no expert is left for has index E and weight 0
             backward: the gradient of x from that of w, the choice held fixed
  combine    y[t] = sum over j of w[t, j] z[t k + j];  dz[t k + j] = w[t, j] dy[t],  dw[t, j] = <dy[t], z[t k + j]>
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one generated token's row: a call whose time is its launch
        {"name": "embed_bf16_token", "op": "embed", "dir": "forward", "dtype": "bf16", "rows": 1, "entries": 32000, "c": 1024, "index": "tokens", "pad": False},
        # 16384 tokens laid out for four experts each
        {"name": "embed_bf16_dispatch", "op": "embed", "dir": "forward", "dtype": "bf16", "rows": 65536, "entries": 16384, "c": 1024, "index": "repeat", "pad": False},
        # gradient of a species-pair table over the 4096-atom frame's edges, whose groups the frame keeps
        {"name": "embed_grad_f32_pairs", "op": "embed", "dir": "backward", "dtype": "f32", "rows": 647170, "entries": 16, "c": 32, "index": "species", "pad": False},
        # a training step's token table: frequencies fall with the rank, padding has no row; sorting is part of the call
        {"name": "embed_grad_bf16_tokens", "op": "embed", "dir": "backward", "dtype": "bf16", "rows": 16384, "entries": 32000, "c": 2048, "index": "tokens", "pad": True},
        # one token between two blocks
        {"name": "norm_bf16_token", "op": "norm", "dir": "forward", "dtype": "bf16", "rows": 1, "c": 1024, "bias": True},
        # sizes that no tile divides, in fp32
        {"name": "norm_f32", "op": "norm", "dir": "forward", "dtype": "f32", "rows": 8191, "c": 777, "bias": True},
        # the largest: gradients of long sequences of wide tokens
        {"name": "norm_grad_bf16_wide", "op": "norm", "dir": "backward", "dtype": "bf16", "rows": 32768, "c": 2048, "bias": True},
        # four tokens of a serving step
        {"name": "route_f32_few", "op": "route", "dir": "forward", "dtype": "f32", "rows": 4, "experts": 64, "k": 2, "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "best": 1, "renormalise": True, "mask": False},
        # a training batch over many experts: sigmoid scores, a bias for balance, groups
        {"name": "route_bf16_groups", "op": "route", "dir": "forward", "dtype": "bf16", "rows": 16384, "experts": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "best": 2, "renormalise": True, "mask": False},
        # gradients where every expert's logit has one, with padding rows and experts switched off
        {"name": "route_grad_f32", "op": "route", "dir": "backward", "dtype": "f32", "rows": 8191, "experts": 160, "k": 6, "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "best": 1, "renormalise": False, "mask": True},
        # the experts' rows of 16384 tokens, four each, back to the tokens
        {"name": "combine_bf16", "op": "combine", "dir": "forward", "dtype": "bf16", "rows": 16384, "k": 4, "c": 1024},
        # their gradients at odd sizes
        {"name": "combine_grad_bf16", "op": "combine", "dir": "backward", "dtype": "bf16", "rows": 8191, "k": 6, "c": 776},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    c = _log(rng, lo, hi)
    return 8 * -(-c // 8) if rng.random() < 0.75 else c   # most widths are multiples of 8


def draw(rng):
    op = rng.choice(["embed", "norm", "route", "route", "combine"])
    case = {"op": op, "dir": rng.choice(["forward", "backward"]), "dtype": rng.choice(["f32", "bf16"])}
    e = 4 if case["dtype"] == "f32" else 2
    if op == "embed":
        c, index = _width(rng, 8, 8192), rng.choice(["tokens", "species", "repeat"])
        rows = _log(rng, 1, min(647170, (96 << 20) // (c * e)))
        entries = _log(rng, 1, 64) if index == "species" else max(1, rows // rng.choice([1, 2, 6, 8])) if index == "repeat" else _log(rng, 64, min(200000, (128 << 20) // (c * e)))
        return {**case, "rows": rows, "entries": entries, "c": c, "index": index, "pad": rng.random() < 0.5}
    if op == "norm":
        c = _width(rng, 8, 8192)
        return {**case, "rows": _log(rng, 1, min(1 << 20, (128 << 20) // (c * e))), "c": c, "bias": rng.random() < 0.7}
    if op == "combine":
        c, k = _width(rng, 8, 8192), _log(rng, 1, 16)
        return {**case, "rows": _log(rng, 1, max(1, min(1 << 18, (128 << 20) // (c * k * e)))), "k": k, "c": c}
    groups = rng.choice([1, 1, 2, 4, 8])
    experts = groups * _log(rng, 2, 512 // groups)
    top_groups = rng.randint(1, groups)
    k = min(_log(rng, 1, 16), experts // groups * top_groups)
    return {**case, "rows": _log(rng, 1, 65536), "experts": experts, "k": k, "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
            "top_groups": top_groups, "best": rng.choice([1, 2]), "renormalise": rng.random() < 0.6, "mask": rng.random() < 0.4}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shares(case):
    """How often each entry is drawn: tokens by the inverse of their rank, species by the root of it."""
    at = torch.arange(1, case["entries"] + 1, dtype=torch.float64)
    return 1 / (at + 2.7) if case["index"] == "tokens" else at ** -0.5


SCALE = 0.7        # of the lookup
WEIGHT_SCALE = 2.5   # of the routing weights


def prepare(case, seed):
    gen = _gen(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    dt, rows, s = DTYPES[case["dtype"]], case["rows"], {"case": case}
    if case["op"] == "embed":
        v, c = case["entries"], case["c"]
        if case["index"] == "repeat":   # row i belongs to token i // k, k rows a token (the last tokens have the rest)
            index = torch.arange(rows, device="cuda") * v // rows
        else:
            rank = torch.randperm(v, generator=gen, device="cuda")   # which entry has which frequency
            cum = _shares(case).cumsum(0).cuda()
            u = torch.rand(rows, generator=gen, device="cuda", dtype=torch.float64) * cum[-1]
            index = rank[torch.searchsorted(cum, u).clamp_(max=v - 1)]
        if case["pad"]:
            index = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.03, -1, index)
        s["index"] = index
        if case["dir"] == "forward":
            s["table"] = normal(v, c, std=0.3, dtype=dt)
        else:
            s["gy"] = normal(rows, c, std=0.1, dtype=dt)
            if case["index"] != "tokens":   # groups that the frame or the router made already
                key = torch.where(index < 0, v, index)
                s["perm"] = torch.sort(key, stable=True)[1].to(torch.int32)
                count = torch.bincount(key, minlength=v + 1)[:v]
                s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)]).to(torch.int32)
        return s
    if case["op"] == "norm":
        c = case["c"]
        s.update(x=normal(rows, c, std=1.5, dtype=dt) + normal(rows, 1, std=0.5).to(dt), w=1 + normal(c, std=0.1), b=normal(c, std=0.1) if case["bias"] else None)
        if case["dir"] == "backward":
            s["gy"] = normal(rows, c, dtype=dt)
        return s
    if case["op"] == "combine":
        k, c = case["k"], case["c"]
        s.update(z=normal(rows * k, c, dtype=dt), weight=torch.softmax(normal(rows, k), 1))
        if case["dir"] == "backward":
            s["gy"] = normal(rows, c, dtype=dt)
        return s
    e, k = case["experts"], case["k"]
    x = normal(rows, e, std=1.3) + normal(e, std=0.5)
    if case["mask"]:
        off = torch.rand(rows, e, generator=gen, device="cuda") < 0.2
        # switched off by -inf or, in a third of the rows, by the type's lowest value; a twentieth of the rows is padding
        lowest = torch.where(torch.arange(rows, device="cuda") % 3 == 0, torch.finfo(dt).min, -math.inf)
        x = torch.where(off, lowest[:, None].float(), x)
        x = torch.where(torch.rand(rows, 1, generator=gen, device="cuda") < 0.05, -math.inf, x)
    s.update(x=x.to(dt), bias=normal(e, std=0.05) if case["bias"] else None)
    if case["dir"] == "backward":
        s["expert"] = _choose(s)
        s["gw"] = normal(rows, k)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------

def _plain_embed(s):
    case, index, v = s["case"], s["index"], s["case"]["entries"]
    inside = (index >= 0) & (index < v)
    if case["dir"] == "forward":
        y = s["table"][torch.where(inside, index, 0)]
        return (torch.where(inside[:, None], y.float(), 0.0) * SCALE).to(y.dtype)
    gy = s["gy"]
    key = torch.where(inside, index, v)
    # sums of many rows in 64 bits; into few entries they are a product with the rows' indicators, not additions to the same few addresses
    wide = torch.float64 if case["rows"] > 64 * v else torch.float32
    if v <= 64:
        parts = max(1, case["rows"] // 1024)   # summed on their own first: one product over all rows keeps few of the card's units busy
        fill = -case["rows"] % parts
        one = torch.cat([key, key.new_full((fill,), v)]).view(parts, 1, -1) == torch.arange(v, device=gy.device)[:, None]
        gy_parts = torch.cat([gy.to(wide), gy.new_zeros((fill, case["c"]), dtype=wide)]).view(parts, -1, case["c"])
        out = torch.bmm(one.to(wide), gy_parts).sum(0)
    else:
        out = torch.zeros(v + 1, case["c"], dtype=wide, device=gy.device).index_add_(0, key, gy.to(wide))[:v]
    return (out * SCALE).to(gy.dtype)


def _plain_norm(s):
    x, w, b = s["x"].float(), s["w"], s["b"]
    d = x - x.mean(1, keepdim=True)
    r = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    xh = d * r
    if s["case"]["dir"] == "forward":
        y = xh * w
        return (y if b is None else y + b).to(s["x"].dtype)
    gy = s["gy"].float()
    t = gy * w
    gx = r * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    out = {"grad_x": gx.to(s["x"].dtype), "grad_w": (gy * xh).sum(0)}
    return out if b is None else {**out, "grad_b": gy.sum(0)}


def _scores(case, x):
    """Scores in 64 bits: what decides between two experts may lie below the last bit of 32."""
    x = x.double()
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def _choose(s):
    """Chosen experts (rows, k) int64, by stable sorts."""
    case, x, bias = s["case"], s["x"], s["bias"]
    m, e, g = x.shape[0], case["experts"], case["groups"]
    key = x.double()
    there = key > -math.inf
    if bias is not None or g > 1:
        q = _scores(case, x)
        if bias is not None:
            q = q + bias.double()
            there = there & (bias > -math.inf)
            key = q
        if g > 1:
            q = torch.where(there, q, -math.inf).view(m, g, e // g)
            best = torch.sort(q, dim=2, descending=True)[0][:, :, :case["best"]]
            score = torch.where(best > -math.inf, best, 0.0).sum(2)
            score = torch.where(best[:, :, 0] > -math.inf, score, -math.inf)
            order = torch.sort(score, dim=1, stable=True, descending=True)[1][:, :case["top_groups"]]
            stay = torch.zeros(m, g, dtype=torch.bool, device=x.device)
            stay.scatter_(1, order, True)
            there = there & stay[:, :, None].expand(m, g, e // g).reshape(m, e)
    key = torch.where(there, key, -math.inf)
    value, order = torch.sort(key, dim=1, stable=True, descending=True)
    return torch.where(value[:, :case["k"]] > -math.inf, order[:, :case["k"]], e)


def _chosen_scores(case, x, expert):
    """(p, s): the slots' shares of their sum and their scores, 64 bits, 0 in empty slots."""
    e = case["experts"]
    live = expert < e
    at = torch.where(live, expert, 0)
    xs = torch.where(live, torch.gather(x.double(), 1, at), -math.inf)
    s = torch.where(live, torch.gather(_scores(case, x), 1, at), 0.0)
    if case["score"] == "softmax":   # the shares from the chosen logits alone: far below the row's largest they still have some
        top = xs.amax(1, keepdim=True)
        p = torch.exp(xs - torch.where(top == -math.inf, 0.0, top))
    else:
        p = s
    total = p.sum(1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), s


def _plain_route(s):
    case, x = s["case"], s["x"]
    if case["dir"] == "forward":
        expert = _choose(s)
        p, sc = _chosen_scores(case, x, expert)
        return {"weight": (WEIGHT_SCALE * (p if case["renormalise"] else sc)).float(), "expert": expert}
    expert, e = s["expert"], case["experts"]
    live = expert < e
    gw = torch.where(live, s["gw"], 0.0) * WEIGHT_SCALE
    p, sc = _chosen_scores(case, x, expert)
    p, sc = p.float(), sc.float()
    if case["renormalise"]:
        g = p * (gw - (gw * p).sum(1, keepdim=True))
        g = g * (1 - sc) if case["score"] == "sigmoid" else g
    elif case["score"] == "sigmoid":
        g = gw * sc * (1 - sc)
    else:
        g = gw * sc
    out = torch.zeros(x.shape[0], e + 1, device=x.device)
    out.scatter_add_(1, expert, g)
    out = out[:, :e]
    if case["score"] == "softmax" and not case["renormalise"]:
        out = out - _scores(case, x).float() * g.sum(1, keepdim=True)
    return out.to(x.dtype)


def _plain_combine(s):
    case, w = s["case"], s["weight"]
    z = s["z"].float().view(case["rows"], case["k"], case["c"])
    if case["dir"] == "forward":
        return (z * w[:, :, None]).sum(1).to(s["z"].dtype)
    gy = s["gy"].float()[:, None, :]
    return {"grad_z": (gy * w[:, :, None]).to(s["z"].dtype).view(-1, case["c"]), "grad_weight": (gy * z).sum(2)}


# ---- the framework's kernels -----------------------------------------------------------------------------------

def _own(s):
    import edge_node_scatter_amd as zs

    case, back = s["case"], s["case"]["dir"] == "backward"
    if case["op"] == "embed":
        if not back:
            return zs.zs_embedding(s["table"], s["index"], scale=SCALE)
        groups = zs.Csr(s["offsets"], s["perm"], None, case["entries"]) if "perm" in s else None
        return zs.zs_embedding_backward(s["gy"], s["index"], case["entries"], scale=SCALE, groups=groups)
    if case["op"] == "norm":
        if not back:
            return zs.zs_layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        gx, gw, gb = zs.zs_layer_norm_backward(s["gy"], s["x"], s["w"], need_b=s["b"] is not None, eps=EPS)
        return {"grad_x": gx, "grad_w": gw} if gb is None else {"grad_x": gx, "grad_w": gw, "grad_b": gb}
    if case["op"] == "combine":
        if not back:
            return zs.zs_combine(s["z"], s["weight"])
        gz, gw = zs.zs_combine_backward(s["gy"], s["z"], s["weight"])
        return {"grad_z": gz, "grad_weight": gw}
    if "router" not in s:   # made once with the model
        s["router"] = zs.Router(case["experts"], case["k"], score=case["score"], groups=case["groups"], top_groups=case["top_groups"], best=case["best"],
                                renormalise=case["renormalise"], scale=WEIGHT_SCALE)
    if back:
        return zs.zs_route_backward(s["gw"], s["x"], s["expert"], s["router"])
    weight, expert = zs.zs_route(s["x"], s["router"], s["bias"])
    return {"weight": weight, "expert": expert}


def run(state):
    if own:
        return _own(state)
    return {"embed": _plain_embed, "norm": _plain_norm, "route": _plain_route, "combine": _plain_combine}[state["case"]["op"]](state)


def _distinct(case):
    """Entries that a lookup reads, on average."""
    if case["index"] == "repeat":
        return min(case["rows"], case["entries"])
    p = _shares(case)
    p = p / p.sum()
    return float((1 - torch.exp(case["rows"] * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


def work(case):
    e, rows, back = 4 if case["dtype"] == "f32" else 2, case["rows"], case["dir"] == "backward"
    if case["op"] == "embed":
        v, c = case["entries"], case["c"]
        if not back:
            return {"bytes": int(e * c * (rows + _distinct(case))) + 8 * rows, "flops": rows * c}
        return {"bytes": e * c * (rows + v) + (8 * rows if case["index"] == "tokens" else 4 * (rows + v + 1)), "flops": c * (rows + v)}
    if case["op"] == "norm":
        c = case["c"]
        b = 1 if case["bias"] else 0
        if not back:
            return {"bytes": 2 * e * rows * c + 4 * c * (1 + b), "flops": 7 * rows * c}
        return {"bytes": 3 * e * rows * c + 4 * c * (2 + b), "flops": 17 * rows * c}
    if case["op"] == "combine":
        c, k = case["c"], case["k"]
        if not back:
            return {"bytes": rows * (e * c * (k + 1) + 4 * k), "flops": 2 * rows * k * c}
        return {"bytes": rows * (e * c * (2 * k + 1) + 8 * k), "flops": 3 * rows * k * c}
    n, k = case["experts"], case["k"]
    bias = 4 * n if case["bias"] else 0
    if not back:
        return {"bytes": rows * (e * n + 12 * k) + bias, "flops": 6 * rows * n}
    # of the logits, all where every expert has a part in the weights, else the chosen ones
    read = n if case["score"] == "softmax" and not case["renormalise"] else k
    return {"bytes": rows * (e * (n + read) + 12 * k), "flops": 6 * rows * read}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------

def _exact_embed(s):
    case, index, v = s["case"], s["index"], s["case"]["entries"]
    if case["dir"] == "forward":
        rows = torch.cat([s["table"].double() * SCALE, torch.zeros(1, case["c"], dtype=torch.float64, device="cuda")])
        return rows[torch.where((index < 0) | (index >= v), v, index)]
    order = torch.argsort(index, stable=True)
    order = order[(index < 0).sum():]
    out = torch.zeros(v, case["c"], dtype=torch.float64, device="cuda")
    # rows in sorted order, and each entry's sum between the places where it starts and ends, a slice of columns at a time
    ends = torch.searchsorted(index[order], torch.arange(v, device="cuda"), right=True)
    begins = torch.searchsorted(index[order], torch.arange(v, device="cuda"))
    for lo in range(0, case["c"], 64):
        part = s["gy"][order, lo:lo + 64].double()
        lengths = (ends - begins)
        out[:, lo:lo + 64] = torch.segment_reduce(part, "sum", lengths=lengths, axis=0, unsafe=True) if part.shape[0] else 0.0
    return out * SCALE


def _exact_norm(s):
    x, w, c = s["x"].double(), s["w"].double(), s["case"]["c"]
    mean = x.sum(1, keepdim=True) / c
    inv = ((x - mean).square().sum(1, keepdim=True) / c + EPS) ** -0.5
    if s["case"]["dir"] == "forward":
        y = (x - mean) * inv * w
        return y if s["b"] is None else y + s["b"].double()
    gy = s["gy"].double()
    u = gy * w
    # through the deviation d = x - mean: y = d inv w, inv = (mean d^2 + eps)^(-1/2)
    d = x - mean
    gd = u * inv - d * inv ** 3 * (u * d).sum(1, keepdim=True) / c
    out = {"grad_x": gd - gd.sum(1, keepdim=True) / c, "grad_w": (gy * d * inv).sum(0)}
    return out if s["b"] is None else {**out, "grad_b": gy.sum(0)}


def _first_best(q):
    """Index of each row's largest entry, the lowest of equal ones."""
    top = q.amax(1, keepdim=True)
    at = torch.arange(q.shape[1], device=q.device)
    return torch.where(q == top, at, q.shape[1]).amin(1)


def _exact_scores(case, x):
    x = x.double()
    if case["score"] == "sigmoid":
        return torch.sigmoid(x)
    empty = (x == -math.inf).all(1, keepdim=True)
    return torch.where(empty, 0.0, torch.softmax(torch.where(empty, 0.0, x), 1))


def _exact_choice(s):
    case, x = s["case"], s["x"].double()
    n, g = case["experts"], case["groups"]
    there = x > -math.inf
    q = _exact_scores(case, x)
    if s["bias"] is not None:
        q = q + s["bias"].double()
        there &= s["bias"] > -math.inf
    q = q.masked_fill(~there, -math.inf)
    if g > 1:
        per = n // g
        parts = []
        for i in range(g):
            part = q[:, i * per:(i + 1) * per].clone()
            total = part.amax(1)
            if case["best"] == 2 and per > 1:
                part.scatter_(1, _first_best(part)[:, None], -math.inf)
                second = part.amax(1)
                total = torch.where(second > -math.inf, total + second, total)
            parts.append(total)
        score = torch.stack(parts, 1)
        keep = torch.zeros_like(score, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            at = _first_best(torch.where(keep, math.nan, score).nan_to_num(nan=-math.inf, neginf=-1e300))
            keep.scatter_(1, at[:, None], True)
        there &= keep.repeat_interleave(per, 1)
    rank = q if s["bias"] is not None else x
    rank = rank.masked_fill(~there, -math.inf)
    out = torch.full((x.shape[0], case["k"]), n, dtype=torch.int64, device="cuda")
    for j in range(case["k"]):
        at = _first_best(rank)
        out[:, j] = torch.where(rank.amax(1) > -math.inf, at, n)
        rank.scatter_(1, at[:, None], -math.inf)
    return out


def _exact_weights(case, x, expert):
    """Weights (rows, k) in 64 bits, differentiable in x."""
    n = case["experts"]
    live = expert < n
    at = expert.clamp(max=n - 1)
    if case["renormalise"]:
        logs = x.gather(1, at)
        if case["score"] == "sigmoid":
            logs = torch.nn.functional.logsigmoid(logs)
        logs = torch.where(live, logs, -math.inf)
        dead = ~live.any(1, keepdim=True)
        w = torch.where(live, torch.softmax(torch.where(dead, 0.0, logs), 1), 0.0)
    else:
        w = torch.where(live, _exact_scores(case, x).gather(1, at), 0.0)
    return WEIGHT_SCALE * w


def _exact_route(s):
    case = s["case"]
    if case["dir"] == "forward":
        expert = _exact_choice(s)
        w = _exact_weights(case, s["x"].double(), expert)
        if case["renormalise"] and case["score"] == "sigmoid":
            # a row whose chosen scores are all 0 in 64 bits has no weights
            some = torch.where(expert < case["experts"], _exact_scores(case, s["x"]).gather(1, expert.clamp(max=case["experts"] - 1)), 0.0).sum(1, keepdim=True)
            w = torch.where(some > 0, w, 0.0)
        return {"weight": w, "expert": expert}
    # the Jacobian's product column by column: dw_j / dx_e by the quotient rule, in 64 bits
    x, expert, n = s["x"].double(), s["expert"], case["experts"]
    w = _exact_weights(case, x, expert) / WEIGHT_SCALE
    gw = torch.where(expert < n, s["gw"].double() * WEIGHT_SCALE, 0.0)
    sc = _exact_scores(case, x)
    own_part = gw * w
    out = torch.zeros(x.shape[0], n + 1, dtype=torch.float64, device="cuda")
    if case["renormalise"]:
        d = own_part - w * own_part.sum(1, keepdim=True)
        if case["score"] == "sigmoid":
            d = d * torch.sigmoid(-torch.cat([x, torch.zeros_like(x[:, :1])], 1).gather(1, expert))
            some = torch.where(expert < n, torch.cat([sc, torch.zeros_like(sc[:, :1])], 1).gather(1, expert), 0.0).sum(1, keepdim=True)
            d = torch.where(some > 0, d, 0.0)
        return out.scatter_add_(1, expert, d)[:, :n]
    if case["score"] == "sigmoid":
        d = own_part * torch.sigmoid(-torch.cat([x, torch.zeros_like(x[:, :1])], 1).gather(1, expert))
        return out.scatter_add_(1, expert, d)[:, :n]
    return out.scatter_add_(1, expert, own_part)[:, :n] - sc * own_part.sum(1, keepdim=True)


def _exact_combine(s):
    case, w = s["case"], s["weight"].double()
    rows, k, c = case["rows"], case["k"], case["c"]
    if case["dir"] == "forward":
        out = torch.zeros(rows, c, dtype=torch.float64, device="cuda")
        for j in range(k):
            out += w[:, j, None] * s["z"][j::k].double()
        return out
    gy = s["gy"].double()
    gz = torch.empty(rows * k, c, dtype=torch.float64, device="cuda")
    gw = torch.empty(rows, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        gz[j::k] = w[:, j, None] * gy
        gw[:, j] = (gy * s["z"][j::k].double()).sum(1)
    return {"grad_z": gz, "grad_weight": gw}


def exact(case, seed):
    return {"embed": _exact_embed, "norm": _exact_norm, "route": _exact_route, "combine": _exact_combine}[case["op"]](prepare(case, seed))
