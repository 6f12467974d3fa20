"""Measured cases of the operators around the scatter: products grouped by species or expert, the gated
residual join between two norms, and the AdamW step over all parameter tensors.

``listed`` and ``draw`` give the cases, ``prepare`` makes a case's inputs on the GPU from a seed, ``run`` does one
pass: the plain form in elementary torch operations where ``own`` is false, the framework's kernels where it is
true.  ``exact`` is the same pass from the definitions in float64.

Definitions (rows i, groups g(i), widths K and N or C, all sums over the named index):

  product    y[i] = x[i] W[g(i)]
             dx[i] = dy[i] W[g(i)]^T,  dW[g] = sum over rows i of group g of x[i]^T dy[i]
  join       u = z (mean z^2 + eps)^(-1/2) w_post,  y = x + scale sigmoid(gate) u,
             h = y (mean y^2 + eps)^(-1/2) w_pre, and the gradients of all six inputs
  AdamW      m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
             p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) (1 - b2^t)^(-1/2) + eps)
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
# AdamW's constants in the cases
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
BLOCK = 256   # elements that share one scale in the 8-bit state; state slices start at multiples of it


def listed():
    return [
        # one 96-atom frame's node features through per-species weights: a call whose time is its launch
        {"name": "mm_f32_atoms", "op": "mm", "dir": "forward", "dtype": "f32", "rows": 96, "groups": 4, "k": 64, "n": 64, "perm": True, "skew": 0.5},
        # radial basis to three radial slots of 32 channels, weights by species pair, the 1000-atom frame's edges
        {"name": "mm_f32_edges", "op": "mm", "dir": "forward", "dtype": "f32", "rows": 158002, "groups": 9, "k": 32, "n": 96, "perm": True, "skew": 1.0},
        # the same products' gradients at the 4096-atom frame's edge count
        {"name": "mm_grad_f32_edges", "op": "mm", "dir": "backward", "dtype": "f32", "rows": 647170, "groups": 16, "k": 32, "n": 96, "perm": True, "skew": 1.0},
        # expert products of a wide block in bf16, rows already sorted by expert
        {"name": "mm_bf16_experts", "op": "mm", "dir": "forward", "dtype": "bf16", "rows": 16384, "groups": 8, "k": 1024, "n": 2048, "perm": False, "skew": 0.5},
        # their gradients at sizes that no tile divides, rows in their own order
        {"name": "mm_grad_bf16_experts", "op": "mm", "dir": "backward", "dtype": "bf16", "rows": 8191, "groups": 16, "k": 776, "n": 1160, "perm": True, "skew": 1.0},
        # one token between two blocks
        {"name": "join_bf16_token", "op": "join", "dir": "forward", "dtype": "bf16", "rows": 1, "c": 1024, "gate": "row"},
        # 4096 nodes of 16 rows, 32 channels
        {"name": "join_f32_nodes", "op": "join", "dir": "forward", "dtype": "f32", "rows": 65536, "c": 32, "gate": "full"},
        # a training step's gradients at a width that is no power of two
        {"name": "join_grad_f32", "op": "join", "dir": "backward", "dtype": "f32", "rows": 16384, "c": 520, "gate": "row"},
        # the largest: long sequences of wide tokens in bf16
        {"name": "join_grad_bf16_wide", "op": "join", "dir": "backward", "dtype": "bf16", "rows": 32768, "c": 2048, "gate": "full"},
        # all tensors of a small network
        {"name": "adamw_32_small", "op": "adamw", "tensors": 24, "total": 60000, "bits": 32, "copy": False},
        # a network of 120 million parameters with bf16 working copies
        {"name": "adamw_32_large", "op": "adamw", "tensors": 28, "total": 120000000, "bits": 32, "copy": True},
        # states in 8 bits, odd tensor sizes
        {"name": "adamw_8", "op": "adamw", "tensors": 30, "total": 24000000, "bits": 8, "copy": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mm", "mm", "join", "adamw"])
    if op == "mm":
        case = {"op": "mm", "dir": rng.choice(["forward", "backward"]), "dtype": rng.choice(["f32", "bf16"]), "perm": rng.random() < 0.5, "skew": round(rng.uniform(0, 1), 2)}
        wide = case["dtype"] == "bf16" and rng.random() < 0.6
        k, n = (_log(rng, 256, 2048), _log(rng, 256, 2048)) if wide else (_log(rng, 8, 256), _log(rng, 8, 256))
        if rng.random() < 0.75:   # most widths are multiples of 8
            k, n = 8 * -(-k // 8), 8 * -(-n // 8)
        groups = _log(rng, 1, 32)
        # no more than the largest listed case moves or computes
        top = min(647170, int(16384 * 1024 * 2048 / (k * n)) if wide else 647170 * 128 // (k + n))
        if case["dir"] == "backward" and wide:
            top //= 2
        rows = _log(rng, 1, max(1, top))
        return {**case, "rows": rows, "groups": groups, "k": k, "n": n}
    if op == "join":
        c = _log(rng, 8, 8192)
        if rng.random() < 0.75:
            c = 8 * -(-c // 8)
        rows = _log(rng, 1, 32768 * 2048 // c if c >= 64 else 1 << 20)
        dtype = rng.choice(["f32", "bf16"])
        return {"op": "join", "dir": rng.choice(["forward", "backward"]), "dtype": dtype, "rows": max(1, rows // 2 if dtype == "f32" else rows), "c": c, "gate": rng.choice(["row", "full"])}
    bits = rng.choice([32, 8])
    return {"op": "adamw", "tensors": _log(rng, 1, 30), "total": _log(rng, 1000, 100000000 if bits == 32 else 24000000), "bits": bits, "copy": rng.random() < 0.5}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _adamw_sizes(case):
    """Tensor sizes of a network: most of the elements in a few products' weights, the others vectors of odd sizes."""
    t, total = case["tensors"], case["total"]
    share = [1.0 if i % 3 == 0 else 0.3 if i % 3 == 1 else 0.002 for i in range(t)]
    return [max(1, int(total * s / sum(share)) + i * i % 7) for i, s in enumerate(share)]


def _group_sizes(case, seed):
    """Rows of each group: weights (j + 1)^-skew in an order drawn from the seed, every eighth group empty."""
    g = case["groups"]
    r = torch.Generator().manual_seed(seed)
    share = torch.arange(1, g + 1, dtype=torch.float64) ** -case["skew"]
    share = share[torch.randperm(g, generator=r)]
    if g >= 8:
        share[3::8] = 0
    at = torch.cat([torch.zeros(1, dtype=torch.float64), share.cumsum(0)]) / share.sum()
    return (at * case["rows"]).round().to(torch.int64)


def prepare(case, seed):
    gen = _gen(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    if case["op"] == "mm":
        dt, rows, k, n, g = DTYPES[case["dtype"]], case["rows"], case["k"], case["n"], case["groups"]
        offsets = _group_sizes(case, seed)
        s = {"case": case, "x": normal(rows, k, dtype=dt), "w": normal(g, k, n, std=k ** -0.5, dtype=dt),
             "offsets": offsets.to(torch.int32).cuda(), "perm": None, "most": max(1, int((offsets[1:] - offsets[:-1]).max()))}
        if case["perm"]:
            # the stable sort of the rows' groups: rows of a group in increasing index
            group = torch.repeat_interleave(torch.arange(g), offsets[1:] - offsets[:-1])
            group = group[torch.randperm(rows, generator=torch.Generator().manual_seed(seed))].cuda()
            s["perm"] = torch.sort(group, stable=True)[1].to(torch.int32)
            s["group"] = group.to(torch.int32)
        if case["dir"] == "backward":
            s["gy"] = normal(rows, n, dtype=dt)
        return s
    if case["op"] == "join":
        dt, rows, c = DTYPES[case["dtype"]], case["rows"], case["c"]
        s = {"case": case, "x": normal(rows, c, dtype=dt), "z": normal(rows, c, std=0.7, dtype=dt),
             "gate": normal(rows, 1 if case["gate"] == "row" else c, std=2.0, dtype=dt),
             "scale": normal(c, std=0.3), "w_post": 1 + normal(c, std=0.1), "w_pre": 1 + normal(c, std=0.1)}
        if case["dir"] == "backward":
            s["gy"], s["gh"] = normal(rows, c, dtype=dt), normal(rows, c, dtype=dt)
        return s
    sizes = _adamw_sizes(case)
    grad_dt = torch.bfloat16 if case["copy"] else torch.float32
    s = {"case": case, "step": 10, "sizes": sizes, "p": [normal(z, std=0.05) for z in sizes],
         "g": [normal(z, std=0.01, dtype=grad_dt) for z in sizes],
         "copy": [torch.zeros(z, dtype=torch.bfloat16, device="cuda") for z in sizes] if case["copy"] else None}
    pads = [-z % BLOCK for z in sizes]
    s["pads"] = pads
    total = sum(sizes) + sum(pads)
    live = torch.cat([torch.arange(z + q, device="cuda") < z for z, q in zip(sizes, pads)])
    m, v = normal(total, std=0.003) * live, normal(total, std=0.004).square() * live
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["seed"] = seed & 0xFFFFFFFF
        s["index"] = torch.cat([torch.arange(z + q, device="cuda") for z, q in zip(sizes, pads)])
        # codes of the starting state (any codes are a valid state) and the scales of its blocks
        s["m_scale"], s["v_scale"] = m.view(-1, BLOCK).abs().amax(1), v.sqrt().view(-1, BLOCK).amax(1)
        sign = (torch.rand(total, generator=gen, device="cuda") < 0.5).to(torch.uint8) * 128
        s["m_code"] = (torch.randint(64, 128, (total,), generator=gen, device="cuda", dtype=torch.uint8) + sign) * live
        s["v_code"] = torch.randint(128, 256, (total,), generator=gen, device="cuda", dtype=torch.uint8) * live
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------

def _padded(s, rows):
    """Rows (M, W) in 32 bits as (G, most, W), each group's rows from the start of its slice, zeros behind."""
    off = s["offsets"].long()
    sorted_rows = rows.float() if s["perm"] is None else rows[s["perm"].long()].float()
    at = torch.arange(rows.shape[0], device=rows.device)
    group = torch.searchsorted(off[1:], at, right=True)
    slot = group * s["most"] + at - off[group]
    out = torch.zeros(s["case"]["groups"] * s["most"], rows.shape[1], device=rows.device)
    out[slot] = sorted_rows
    return out.view(s["case"]["groups"], s["most"], rows.shape[1]), slot


def _rows(s, padded, slot, dtype):
    """The padded rows back in the rows' own order, rounded once."""
    y = padded.reshape(-1, padded.shape[2])[slot].to(dtype)
    if s["perm"] is None:
        return y
    out = torch.empty_like(y)
    out[s["perm"].long()] = y
    return out


def _plain_mm(s):
    x, w = s["x"], s["w"]
    xp, slot = _padded(s, x)
    if s["case"]["dir"] == "forward":
        return _rows(s, torch.bmm(xp, w.float()), slot, x.dtype)
    gp, slot = _padded(s, s["gy"])
    gx = _rows(s, torch.bmm(gp, w.float().transpose(1, 2).contiguous()), slot, x.dtype)
    return {"grad_x": gx, "grad_w": torch.bmm(xp.transpose(1, 2).contiguous(), gp).to(w.dtype)}


def _join_parts(s):
    x, z, a = s["x"].float(), s["z"].float(), s["gate"].float()
    rz = 1 / torch.sqrt((z * z).mean(1, keepdim=True) + EPS)
    sig = 1 / (1 + torch.exp(-a))
    zn = z * rz
    u = zn * s["w_post"]
    y = x + s["scale"] * sig * u
    ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
    return z, rz, sig, zn, u, y, ry


def _plain_join(s):
    dt = s["x"].dtype
    z, rz, sig, zn, u, y, ry = _join_parts(s)
    if s["case"]["dir"] == "forward":
        return {"y": y.to(dt), "h": (y * ry * s["w_pre"]).to(dt)}
    gh = s["gh"].float()
    yn = y * ry
    t = gh * s["w_pre"]
    gy = s["gy"].float() + ry * (t - yn * (t * yn).mean(1, keepdim=True))
    b = gy * sig
    q = b * s["scale"]
    ga = gy * s["scale"] * u * (sig * (1 - sig))
    if s["gate"].shape[1] == 1:
        ga = ga.sum(1, keepdim=True)
    r = q * s["w_post"]
    gz = rz * (r - zn * (r * zn).mean(1, keepdim=True))
    return {"grad_x": gy.to(dt), "grad_z": gz.to(dt), "grad_gate": ga.to(dt), "grad_scale": (b * u).sum(0), "grad_w_post": (q * zn).sum(0),
            "grad_w_pre": (gh * yn).sum(0)}


def _flat(parts, pads):
    gap = torch.zeros(BLOCK, device="cuda")
    return torch.cat([t for x, q in zip(parts, pads) for t in (x.reshape(-1).float(), gap[:q])])


def _split(flat, s):
    cut = [w for z, q in zip(s["sizes"], s["pads"]) for w in (z, q)]
    return list(flat.split(cut)[::2])


# The 8-bit state.  A block's values t = |value| / scale lie in [0, 1]; a code c > 0 stands for the float whose bit
# pattern is (c + base) << shift, so codes are evenly spaced within each power of two and the top code is 1.0.
# m: a sign bit and 7 bits (8 steps a power of two); sqrt(v): 8 bits (16 steps).  Rounding is stochastic, by the
# bits of a hash of the element's index and the step's seed added below the kept bits.
M_SHIFT, M_TOP, V_SHIFT, V_TOP = 20, 127, 19, 255
ONE = 0x3F800000
TINY = 2.0 ** -120


def _hash(index, seed):
    """32 pseudo-random bits: a multiplicative step by 2^32 over the golden ratio and the murmur3 finaliser."""
    h = (index * 0x9E3779B9 + seed) & 0xFFFFFFFF
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _decode(code, shift, top, scale):
    bits = torch.where(code > 0, (code + (ONE >> shift) - top) << shift, 0).to(torch.int32)
    return (bits.view(torch.float32).view(-1, BLOCK) * scale[:, None]).view(-1)


def _encode(mag, shift, top, random, floor):
    """(codes, scales) of non-negative magnitudes."""
    scale = mag.view(-1, BLOCK).amax(1)
    scale = torch.where(scale < TINY, 0.0, scale)
    inv = torch.where(scale > 0, 1 / scale, torch.where(scale == 0, 0.0, scale))
    t = (mag.view(-1, BLOCK) * inv[:, None]).view(-1)
    t = torch.where(t > 1, 1.0, t)
    code = ((t.view(torch.int32).long() + random) >> shift) - ((ONE >> shift) - top)
    return torch.where(t > 0, code.clamp(floor, top), 0), scale


def _plain_adamw(s):
    s["step"] += 1
    t = s["step"]
    p, g = _flat(s["p"], s["pads"]), _flat(s["g"], s["pads"])
    if s["case"]["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        mc, vc = s["m_code"].long(), s["v_code"].long()
        m = _decode(mc & 127, M_SHIFT, M_TOP, s["m_scale"])
        m = torch.where(mc >= 128, -m, m)
        r = _decode(vc, V_SHIFT, V_TOP, s["v_scale"])
        v = r * r
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = torch.sqrt(v)
    p = p * (1 - LR * DECAY) - m / (root * (1 - BETA2 ** t) ** -0.5 + ADAM_EPS) * (LR / (1 - BETA1 ** t))
    s["p"] = _split(p, s)
    out = {"p": s["p"]}
    if s["copy"] is not None:
        s["copy"] = out["copy"] = [x.to(torch.bfloat16) for x in s["p"]]
    if s["case"]["bits"] == 32:
        s["m"], s["v"] = m, v
        return {**out, "m": m, "v": v}
    h = _hash(s["index"], (s["seed"] + t) & 0xFFFFFFFF)
    mc, s["m_scale"] = _encode(m.abs(), M_SHIFT, M_TOP, h & ((1 << M_SHIFT) - 1), 0)
    vc, s["v_scale"] = _encode(root, V_SHIFT, V_TOP, h >> (32 - V_SHIFT), 1)
    s["m_code"], s["v_code"] = (mc + torch.where(m < 0, 128, 0)).to(torch.uint8), vc.to(torch.uint8)
    m = torch.where(m < 0, -_decode(mc, M_SHIFT, M_TOP, s["m_scale"]), _decode(mc, M_SHIFT, M_TOP, s["m_scale"]))
    r = _decode(vc, V_SHIFT, V_TOP, s["v_scale"])
    return {**out, "m": m, "v": r * r}


# ---- the framework's kernels -----------------------------------------------------------------------------------

def _own(s):
    import edge_node_scatter_amd as zs

    case = s["case"]
    if case["op"] == "mm":
        groups = zs.Csr(s["offsets"], s["perm"], None, case["groups"])
        if case["dir"] == "forward":
            return zs.zs_grouped_mm(s["x"], s["w"], groups)
        gx, gw = zs.zs_grouped_mm_backward(s["gy"], s["x"], s["w"], groups)
        return {"grad_x": gx, "grad_w": gw}
    if case["op"] == "join":
        args = (s["x"], s["z"], s["gate"], s["scale"], s["w_post"], s["w_pre"])
        if case["dir"] == "forward":
            y, h = zs.zs_block_join(*args, eps=EPS)
            return {"y": y, "h": h}
        gx, gz, ga, gs, gpost, gpre = zs.zs_block_join_backward(s["gy"], s["gh"], *args, eps=EPS)
        return {"grad_x": gx, "grad_z": gz, "grad_gate": ga, "grad_scale": gs, "grad_w_post": gpost, "grad_w_pre": gpre}
    if "opt" not in s:   # the optimizer that a training program makes once and keeps
        state = {"m": s["m"], "v": s["v"]} if case["bits"] == 32 else {k: s[k] for k in ("m_code", "v_code", "m_scale", "v_scale", "seed")}
        s["opt"] = zs.AdamW(s["p"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=DECAY, state_bits=case["bits"], copies=s["copy"],
                            state={"step": s["step"], **state})
    opt = s["opt"]
    opt.step(s["g"])
    m, v = opt.moments()
    out = {"p": s["p"], "m": m, "v": v}
    return out if s["copy"] is None else {**out, "copy": s["copy"]}


def run(state):
    if own:
        return _own(state)
    return {"mm": _plain_mm, "join": _plain_join, "adamw": _plain_adamw}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "mm":
        e, rows, k, n, g = 2 if case["dtype"] == "bf16" else 4, case["rows"], case["k"], case["n"], case["groups"]
        index = 4 * (g + 1) + (4 * rows if case["perm"] else 0)
        if case["dir"] == "forward":
            return {"bytes": e * (rows * (k + n) + g * k * n) + index, "flops": 2 * rows * k * n}
        return {"bytes": e * (rows * (2 * k + n) + 2 * g * k * n) + index, "flops": 4 * rows * k * n}
    if case["op"] == "join":
        e, rows, c = 2 if case["dtype"] == "bf16" else 4, case["rows"], case["c"]
        a = c if case["gate"] == "full" else 1
        if case["dir"] == "forward":
            return {"bytes": e * rows * (4 * c + a) + 12 * c, "flops": 14 * rows * c}
        return {"bytes": e * rows * (6 * c + 2 * a) + 24 * c, "flops": 45 * rows * c}
    n = sum(_adamw_sizes(case))
    grad, copy = (2, 2) if case["copy"] else (4, 0)
    # p read and written, g read, copy written, states read and written; 8-bit states also come back as values
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
    return {"bytes": n * (8 + grad + copy + state), "flops": 16 * n}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------

def _exact_mm(s):
    case, off = s["case"], s["offsets"].tolist()
    x, w = s["x"].double(), s["w"].double()
    back = case["dir"] == "backward"
    gy = s["gy"].double() if back else None
    y = torch.zeros(case["rows"], case["k" if back else "n"], dtype=torch.float64, device="cuda")
    gw = torch.zeros_like(w)
    for g in range(case["groups"]):
        at = torch.arange(off[g], off[g + 1], device="cuda")
        if s["perm"] is not None:
            at = s["perm"].long()[at]
        if back:
            y[at] = gy[at] @ w[g].T.contiguous()
            gw[g] = x[at].T.contiguous() @ gy[at]
        else:
            y[at] = x[at] @ w[g]
    return {"grad_x": y, "grad_w": gw} if back else y


def _exact_join(s):
    x, z, a, c = s["x"].double(), s["z"].double(), s["gate"].double(), s["case"]["c"]
    scale, post, pre = s["scale"].double(), s["w_post"].double(), s["w_pre"].double()
    zi = (z.square().sum(1, keepdim=True) / c + EPS) ** -0.5
    gate = torch.sigmoid(a)
    y = x + scale * gate * post * z * zi
    yi = (y.square().sum(1, keepdim=True) / c + EPS) ** -0.5
    if s["case"]["dir"] == "forward":
        return {"y": y, "h": pre * y * yi}
    gy, gh = s["gy"].double(), s["gh"].double()
    dy = gy + pre * gh * yi - y * yi ** 3 * (pre * gh * y).sum(1, keepdim=True) / c
    du = dy * scale * gate * post
    dz = du * zi - z * zi ** 3 * (du * z).sum(1, keepdim=True) / c
    da = dy * scale * post * z * zi * gate * (1 - gate)
    return {"grad_x": dy, "grad_z": dz, "grad_gate": da.sum(1, keepdim=True) if a.shape[1] == 1 else da, "grad_scale": (dy * gate * post * z * zi).sum(0),
            "grad_w_post": (dy * scale * gate * z * zi).sum(0), "grad_w_pre": (gh * y * yi).sum(0)}


def _exact_adamw(s):
    t, sizes, starts = s["step"] + 1, s["sizes"], []
    at = 0
    for z, q in zip(sizes, s["pads"]):
        starts.append(at)
        at += z + q
    total = at

    def value(code, levels, steps):   # 2^(octave) (1 + fraction), the top code being 1
        down = levels - code
        octave = -torch.div(down + steps - 1, steps, rounding_mode="floor")
        return torch.where(code > 0, torch.exp2(octave.double()) * (1 + ((-down) % steps).double() / steps), 0.0)

    if s["case"]["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        mc, vc = s["m_code"].long(), s["v_code"].long()
        each = torch.arange(total, device="cuda") // BLOCK
        m = value(mc % 128, 127, 8) * s["m_scale"].double()[each] * torch.where(mc >= 128, -1.0, 1.0)
        v = (value(vc, 255, 16) * s["v_scale"].double()[each]) ** 2
    new_p = []
    for i, z in enumerate(sizes):
        at = slice(starts[i], starts[i] + z)
        g = s["g"][i].double()
        m[at] = BETA1 * m[at] + (1 - BETA1) * g
        v[at] = BETA2 * v[at] + (1 - BETA2) * g.square()
        hat = (m[at] / (1 - BETA1 ** t)) / ((v[at] / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
        new_p.append(s["p"][i].double() * (1 - LR * DECAY) - LR * hat)
    # the 8-bit states' values after their random rounding depend on each code's last bit in 32-bit arithmetic
    out = {"p": new_p, "m": m if s["case"]["bits"] == 32 else None, "v": v if s["case"]["bits"] == 32 else None}
    return out if s["copy"] is None else {**out, "copy": new_p}


def exact(case, seed):
    return {"mm": _exact_mm, "join": _exact_join, "adamw": _exact_adamw}[case["op"]](prepare(case, seed))
