"""The gated residual join between two norms, and its gradients, against float64 on the GPU."""
import pytest
import torch

import blockref
import edge_node_scatter_amd as zs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.load()
    return torch.device("cuda:0")


def say(*a):
    print("[gpu]", *a, flush=True)


def make(M, c, dtype, gate, seed):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {"x": mk(M, c).to(dtype), "z": (0.7 * mk(M, c)).to(dtype),
         "gate": None if gate is None else (2 * mk(M, 1 if gate == "row" else c)).to(dtype),
         "scale": 0.5 * mk(c), "w_post": 1 + 0.1 * mk(c), "w_pre": 1 + 0.1 * mk(c)}
    return d, mk(M, c).to(dtype), mk(M, c).to(dtype)


NAMES = ("x", "z", "gate", "scale", "w_post", "w_pre")


def on(d, dev):
    return [None if d[k] is None else d[k].to(dev) for k in NAMES]


def reference_grads(d, gy, gh, eps=EPS):
    """Gradients of sum(gy y) + sum(gh h) by float64 autograd of the definition."""
    leaf = {k: None if d[k] is None else d[k].double().requires_grad_() for k in NAMES}
    y, h = blockref.join(*(leaf[k] for k in NAMES), eps)
    loss = (gy.double() * y).sum() if gy is not None else 0
    if h is not None and gh is not None:
        loss = loss + (gh.double() * h).sum()
    live = [leaf[k] for k in NAMES if leaf[k] is not None]
    grads = iter(torch.autograd.grad(loss, live, allow_unused=True))
    out = []
    for k in NAMES:
        g = None if leaf[k] is None else next(grads)
        out.append(torch.zeros_like(leaf[k]) if g is None and leaf[k] is not None else g)
    return out


def close(got, ref, what, dtype, terms, floor=None):
    """Entries are fp32 expressions of about 40 operations whose sums run over `terms` entries of comparable size:
    errors of (40 + 2 sqrt(terms)) fp32 ulps of the array's typical size (its row's, or its own), then one rounding.
    2 sqrt(terms) allows for the random walk of a sum's roundings four standard deviations wide."""
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what
    size = floor if floor is not None else (ref.square().mean(-1, keepdim=True).sqrt() if ref.dim() > 1 else ref.square().mean().sqrt())
    inner = (40 + 2 * terms ** 0.5) * 2.0 ** -23 * (size + ref.abs())
    bound = inner + blockref.ULP[dtype] * (ref.abs() + inner) + 1e-38
    worst = ((got - ref).abs() / bound).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"


WIDTHS = [3, 8, 9, 16, 24, 32, 57, 64, 100, 128, 256, 264, 500, 512, 520, 776, 1000, 1024, 1032, 1536, 2048, 2056, 4096, 4100, 8192]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", WIDTHS)
@pytest.mark.parametrize("gate", [None, "row", "full"])
def test_forward_and_gradients(dev, dtype, c, gate):
    M = 37 if c > 64 else 300
    say("join", M, c, dtype, gate)
    d, gy, gh = make(M, c, dtype, gate, seed=c)
    y, h = zs.zs_block_join(*on(d, dev), eps=EPS)
    ry, rh = blockref.join(*(d[k] for k in NAMES), EPS)
    close(y, ry, "y", dtype, c)
    close(h, rh, "h", dtype, c)
    got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=EPS)
    ref = reference_grads(d, gy, gh)
    for name, g, r in zip(NAMES, got, ref):
        if r is None:
            assert g is None
        elif name == "gate" and gate == "row":
            # a sum over the channels: its typical size is sqrt(c) of an entry's
            full = dict(d, gate=d["gate"].expand(M, c).clone())
            entry = reference_grads(full, gy, gh)[2].abs().sum(1, keepdim=True)
            close(g, r, "grad_gate", dtype, c, floor=entry)
        elif name in ("scale", "w_post", "w_pre"):
            # a sum over the rows
            close(g, r, "grad_" + name, F32, M * 4, floor=torch.full((1,), float(M) ** 0.5, dtype=torch.float64) * r.abs().max().clamp(min=1))
        else:
            close(g, r, "grad_" + name, dtype, c)
    again = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=EPS)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [None, "row"])
def test_one_channel(dev, dtype, gate):
    """The norm of one channel is its sign: gradients through it are what remains of terms of size |t| ry that cancel
    but for eps, so their error is some ulps of those terms, not of themselves."""
    say("one channel", dtype, gate)
    d, gy, gh = make(300, 1, dtype, gate, seed=1)
    y, h = zs.zs_block_join(*on(d, dev), eps=EPS)
    ry, rh = blockref.join(*(d[k] for k in NAMES), EPS)
    close(y, ry, "y", dtype, 1)
    close(h, rh, "h", dtype, 1)
    got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=EPS)
    ref = reference_grads(d, gy, gh)
    term_y = gh.double().abs() * d["w_pre"].double().abs() / torch.sqrt(ry * ry + EPS)
    term_x = gy.double().abs() + term_y
    s = 1.0 if gate is None else torch.sigmoid(d["gate"].double())
    inverse = 1 / torch.sqrt(d["z"].double() ** 2 + EPS)
    term_z = term_x * (d["scale"] * d["w_post"]).double().abs() * s * inverse
    for name, g, r, term in (("x", got[0], ref[0], term_x), ("z", got[1], ref[1], term_z)):
        bound = 42 * 2.0 ** -23 * term + blockref.ULP[dtype] * (r.abs() + 42 * 2.0 ** -23 * term)
        assert ((g.double().cpu() - r).abs() <= bound).all(), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [0, 1, 2, 5, 2049])
def test_row_counts(dev, dtype, M):
    say("rows", M, dtype)
    d, gy, gh = make(M, 48, dtype, "full", seed=M)
    y, h = zs.zs_block_join(*on(d, dev), eps=EPS)
    ry, rh = blockref.join(*(d[k] for k in NAMES), EPS)
    close(y, ry, "y", dtype, 48)
    close(h, rh, "h", dtype, 48)
    got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=EPS)
    if M == 0:
        assert all((g == 0).all() for g in got[3:]) and got[0].shape == (0, 48)
        return
    ref = reference_grads(d, gy, gh)
    for name, g, r in list(zip(NAMES, got, ref))[3:]:
        close(g, r, "grad_" + name, F32, M * 4, floor=torch.full((1,), float(M) ** 0.5, dtype=torch.float64) * r.abs().max().clamp(min=1))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_parts_left_out(dev, dtype):
    """No norm behind (w_pre None), no block (z None), and gradients of one output only."""
    say("parts", dtype)
    d, gy, gh = make(50, 72, dtype, "row", seed=2)
    last = dict(d, w_pre=None)
    y, h = zs.zs_block_join(*on(last, dev), eps=EPS)
    assert h is None
    close(y, blockref.join(*(last[k] for k in NAMES), EPS)[0], "y", dtype, 72)
    got = zs.zs_block_join_backward(gy.to(dev), None, *on(last, dev), eps=EPS)
    ref = reference_grads(last, gy, None)
    assert got[5] is None
    close(got[0], ref[0], "grad_x", dtype, 72)
    close(got[1], ref[1], "grad_z", dtype, 72)
    first = dict(x=d["x"], z=None, gate=None, scale=None, w_post=None, w_pre=d["w_pre"])
    y, h = zs.zs_block_join(*on(first, dev), eps=EPS)
    close(h, blockref.join(*(first[k] for k in NAMES), EPS)[1], "norm", dtype, 72)
    got = zs.zs_block_join_backward(None, gh.to(dev), *on(first, dev), eps=EPS)
    ref = reference_grads(first, None, gh)
    close(got[0], ref[0], "grad_x of the norm", dtype, 72)
    assert got[1] is None and got[3] is None
    close(got[5], ref[5], "grad_w_pre", F32, 200, floor=torch.full((1,), 50.0 ** 0.5, dtype=torch.float64) * ref[5].abs().max())
    for a, b in ((gy, None), (None, gh)):
        got = zs.zs_block_join_backward(*(None if t is None else t.to(dev) for t in (a, b)), *on(d, dev), eps=EPS)
        ref = reference_grads(d, a, b)
        close(got[0], ref[0], "grad_x of one output", dtype, 72)
        close(got[1], ref[1], "grad_z of one output", dtype, 72)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_at_the_ends(dev, dtype):
    """Gates of -inf, the type's lowest and highest values, +inf: factor 0 or 1, gradient of the gate 0, no NaN; a NaN
    gate spoils its own entries."""
    say("gate ends", dtype)
    M, c = 6, 40
    d, gy, gh = make(M, c, dtype, "full", seed=4)
    ends = [float("-inf"), torch.finfo(dtype).min, -200.0, 200.0, torch.finfo(dtype).max, float("inf")]
    for i, e in enumerate(ends):
        d["gate"][i] = e
    y, h = zs.zs_block_join(*on(d, dev), eps=EPS)
    assert torch.equal(y[:3].cpu(), d["x"][:3])
    open_ = dict(d, gate=None)
    ry, rh = blockref.join(*(open_[k] for k in NAMES), EPS)
    close(y[3:], ry[3:], "y of open gates", dtype, c)
    got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=EPS)
    assert all(torch.isfinite(g).all() for g in got)
    assert (got[2][[0, 1, 4, 5]] == 0).all() and (got[1][:3].abs() <= 1e-30).all()
    d["gate"][2, 5] = float("nan")
    y, h = zs.zs_block_join(*on(d, dev), eps=EPS)
    assert torch.isnan(y[2, 5]) and torch.isfinite(y[2, :5]).all() and torch.isnan(h[2]).all()
    keep = [0, 1, 3, 4, 5]
    assert torch.isfinite(y[keep]).all() and torch.isfinite(h[keep]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_zero_rows(dev, dtype):
    """Rows of zeros (a masked token) give zeros and finite gradients."""
    say("zero rows", dtype)
    d, gy, gh = make(9, 64, dtype, "full", seed=6)
    d["x"][4], d["z"][4] = 0, 0
    y, h = zs.zs_block_join(*on(d, dev), eps=EPS)
    assert (y[4] == 0).all() and (h[4] == 0).all()
    got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=EPS)
    assert all(torch.isfinite(g).all() for g in got)
    ref = reference_grads(d, gy, gh)
    close(got[0], ref[0], "grad_x", dtype, 64)
    close(got[1], ref[1], "grad_z", dtype, 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [1, 8])
def test_strided_views(dev, dtype, pad):
    say("strided", dtype, pad)
    M, c = 65, 96
    d, gy, gh = make(M, c, dtype, "full", seed=8)
    want = zs.zs_block_join(*on(d, dev), eps=EPS)
    wide = []
    for k in ("x", "z", "gate"):
        b = torch.full((M, c + 2 * pad), float("nan"), dtype=dtype, device=dev)
        b[:, pad:pad + c] = d[k].to(dev)
        wide.append(b[:, pad:pad + c])
    rest = [d[k].to(dev) for k in ("scale", "w_post", "w_pre")]
    got = zs.zs_block_join(*wide, *rest, eps=EPS)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    want = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=EPS)
    got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *wide, *rest, eps=EPS)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_past_32_bits(dev, dtype):
    """Row strides that take rows more than 2^32 elements from the start."""
    M, c, stride = 260, 64, 1 << 25
    say("wide offsets", dtype)
    d, gy, gh = make(M, c, dtype, "full", seed=31)
    big = torch.empty((M - 1) * stride + c, dtype=dtype, device=dev)
    assert big.numel() > 1 << 32
    args = on(d, dev)
    want = zs.zs_block_join(*args, eps=EPS)
    back = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *args, eps=EPS)
    for i in range(3):
        view = big.as_strided((M, c), (stride, 1))
        view.copy_(args[i])
        wide = [view if j == i else t for j, t in enumerate(args)]
        assert all(torch.equal(a, b) for a, b in zip(want, zs.zs_block_join(*wide, eps=EPS)))
        got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *wide, eps=EPS)
        assert all(torch.equal(a, b) for a, b in zip(back, got))


def test_autograd_against_differences(dev):
    """block_join and block_norm under autograd: a directional derivative against central differences in float64."""
    say("autograd")
    M, c = 40, 56
    d, gy, gh = make(M, c, F32, "row", seed=12)
    leaves = [t.requires_grad_() for t in on(d, dev)]
    y, h = zs.block_join(*leaves, eps=EPS)
    ((y * gy.to(dev)).sum() + (h * gh.to(dev)).sum()).backward()
    gen = torch.Generator().manual_seed(0)
    dirs = [torch.randn(d[k].shape, generator=gen).double() for k in NAMES]

    def f(t):
        y, h = blockref.join(*(d[k].double() + t * v for k, v in zip(NAMES, dirs)), EPS)
        return ((gy.double() * y).sum() + (gh.double() * h).sum()).item()

    step = 1e-4   # the difference's own error: step^2 times third derivatives of order of the sum's terms
    slope = (f(step) - f(-step)) / (2 * step)
    parts = [(t.grad.double().cpu() * v) for t, v in zip(leaves, dirs)]
    got, size = sum(p.sum().item() for p in parts), sum(p.abs().sum().item() for p in parts)
    assert abs(got - slope) <= 1e-5 * size
    x = d["x"].to(dev).requires_grad_()
    w = d["w_pre"].to(dev).requires_grad_()
    zs.block_norm(x, w, EPS).sum().backward()
    assert torch.isfinite(x.grad).all() and torch.isfinite(w.grad).all()
    only_y = zs.block_join(*leaves, eps=EPS)[0]
    g = torch.autograd.grad(only_y.sum(), leaves[0])[0]
    assert torch.equal(g, torch.ones_like(g))


def test_graph_replays(dev):
    say("graph")
    d, gy, gh = make(500, 128, BF16, "full", seed=15)
    args = on(d, dev)
    gyd, ghd = gy.to(dev), gh.to(dev)
    run = lambda: (*zs.zs_block_join(*args, eps=EPS), *zs.zs_block_join_backward(gyd, ghd, *args, eps=EPS))  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run()
    for i in range(4):
        args[0].add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(), res)), i


def test_refusals(dev):
    say("refusals")
    d, gy, gh = make(4, 16, F32, "full", seed=1)
    x, z, gate, scale, post, pre = on(d, dev)
    for bad in ((x.cpu(), z, gate, scale, post, pre), (x, z[:3], gate, scale, post, pre), (x, z, gate[:, :7], scale, post, pre),
                (x, z, gate, scale[:8], post, pre), (x, z, gate, None, post, pre), (x, None, gate, None, None, pre),
                (x, None, None, None, None, None), (x[0], z, gate, scale, post, pre)):
        with pytest.raises(ValueError):
            zs.zs_block_join(*bad)
    with pytest.raises(TypeError):
        zs.zs_block_join(x, z.bfloat16(), gate, scale, post, pre)
    with pytest.raises(TypeError):
        zs.zs_block_join(x, z, gate, scale.bfloat16(), post, pre)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(zs.ZsError):
            zs.zs_block_join(x, z, gate, scale, post, pre, eps=eps)
    wide = torch.zeros(1, 8193, device=dev)
    with pytest.raises(zs.ZsError):
        zs.zs_block_join(wide, None, None, None, None, torch.ones(8193, device=dev))
    with pytest.raises(ValueError):
        zs.zs_block_join_backward(gy.to(dev)[:2], None, x, z, gate, scale, post, pre)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [None, "row", "full"])
@pytest.mark.parametrize("shape", [(5, 16), (37, 48), (300, 57), (301, 264), (6, 520), (37, 1032), (3, 4100)])
def test_small_eps(dev, dtype, gate, shape):
    """eps = 1e-30: rows of zeros in x, in z and in both, whose norms' factor is 1e15, among ordinary rows, and row
    counts that leave the last workgroup part empty."""
    M, c = shape
    say("small eps", M, c, dtype, gate)
    d, gy, gh = make(M, c, dtype, gate, seed=M + c)
    d["x"][M // 2], d["z"][M // 2] = 0, 0
    d["z"][0] = 0
    got = zs.zs_block_join_backward(gy.to(dev), gh.to(dev), *on(d, dev), eps=1e-30)
    ref = reference_grads(d, gy, gh, 1e-30)
    close(got[0], ref[0], "grad_x", dtype, c)
    close(got[1], ref[1], "grad_z", dtype, c)
    for name, g, r in list(zip(NAMES, got, ref))[3:]:
        close(g, r, "grad_" + name, F32, M * 4, floor=torch.full((1,), float(M) ** 0.5, dtype=torch.float64) * r.abs().max())
    first = dict(x=d["x"], z=None, gate=None, scale=None, w_post=None, w_pre=d["w_pre"])
    got = zs.zs_block_join_backward(None, gh.to(dev), *on(first, dev), eps=1e-30)
    ref = reference_grads(first, None, gh, 1e-30)
    close(got[0], ref[0], "grad_x of the norm", dtype, c)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [None, "row", "full"])
@pytest.mark.parametrize("c, size", [(48, 1e-14), (48, 1e12), (48, 1e14), (48, 1e15), (520, 1e16), (1032, 1e16), (520, 1e17), (48, 1e18)])
def test_rows_of_any_size(dev, dtype, gate, c, size):
    """Rows far from 1: the gradient through the norm is a difference of terms of the size 1 / |y|, whatever powers of
    |y| lie between.  Gradients of h alone (grad_y zeros, or none), since grad_y would hide theirs."""
    M = 21
    say("row size", c, dtype, gate, size)
    d, _, gh = make(M, c, dtype, gate, seed=c)
    d["x"] = (d["x"].float() * size).to(dtype)
    if size < 1:
        d["z"] = (d["z"].float() * size).to(dtype)
    eps = 1e-30 if size < 1 else EPS
    ref = reference_grads(d, None, gh, eps)
    for gy in (torch.zeros(M, c, dtype=dtype), None):
        got = zs.zs_block_join_backward(None if gy is None else gy.to(dev), gh.to(dev), *on(d, dev), eps=eps)
        close(got[0], ref[0], "grad_x", dtype, c)
        close(got[1], ref[1], "grad_z", dtype, c)
        for name, g, r in list(zip(NAMES, got, ref))[3:]:
            close(g, r, "grad_" + name, F32, M * 4, floor=torch.full((1,), float(M) ** 0.5, dtype=torch.float64) * r.abs().max())


def test_without_a_block_y_is_x(dev):
    x, w = torch.randn(6, 16, device=dev), torch.ones(16, device=dev)
    for t in (x, x.t().contiguous().t(), torch.randn(6, 20, device=dev)[:, :16]):
        y, h = zs.zs_block_join(t, None, None, None, None, w, eps=EPS)
        assert y is t and h.shape == t.shape
