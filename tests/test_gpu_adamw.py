"""The AdamW step over many tensors, 32- and 8-bit moments, on the GPU against float64."""
import pytest
import torch

import blockref
import edge_node_scatter_amd as zs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HP = dict(lr=2e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.05)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.load()
    return torch.device("cuda:0")


def say(*a):
    print("[gpu]", *a, flush=True)


SETS = {"one": [1], "odd": [1, 3, 4, 5, 255, 256, 257, 1000, 4096, 4099], "many": [(i * 37) % 513 + 1 for i in range(150)],
        "large": [3_000_001, 7, 65536], "with_empty": [0, 5, 0, 300, 0]}


def tensors(sizes, seed, dev, dtype=F32, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=gen) * std).to(dtype).to(dev) for s in sizes]


def slices(opt, flat):
    return [flat[o:o + p.numel()] for o, p in zip(opt.offsets, opt.params)]


def near(got, ref, ulps, what):
    got = got.double().cpu()
    bound = ulps * 2.0 ** -24 * ref.abs() + 1e-37
    bad = ((got - ref).abs() > bound).sum().item()
    assert bad == 0, f"{what}: {bad} of {ref.numel()} outside {ulps} half ulps"


@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("grad_dtype", [F32, BF16])
@pytest.mark.parametrize("copy", [False, True])
def test_32_bit_steps(dev, name, grad_dtype, copy):
    """Five steps; after each, moments within their few roundings of float64 from the same start, parameters within
    the roundings of a chain of nine operations."""
    sizes = SETS[name]
    say("adamw 32", name, grad_dtype, copy)
    params = tensors(sizes, 1, dev)
    copies = [torch.full_like(p, 9, dtype=BF16) for p in params] if copy else None
    opt = zs.AdamW(params, copies=copies, **HP)
    for step in range(1, 6):
        grads = tensors(sizes, 100 + step, dev, grad_dtype, 0.1)
        before = [p.clone() for p in params]
        m0, v0 = ([t.clone() for t in slices(opt, f)] for f in opt.moments())
        opt.step(grads)
        m1, v1 = (slices(opt, f) for f in opt.moments())
        for i, p in enumerate(params):
            rp, rm, rv = blockref.adamw(before[i].cpu(), grads[i].cpu(), m0[i].cpu(), v0[i].cpu(), HP["lr"], *HP["betas"], HP["eps"], HP["weight_decay"], step)
            # m: two products and a sum, constants off by half an ulp; cancellation is relative to the terms
            size = (m0[i].double().abs().cpu() * 0.9 + grads[i].double().abs().cpu() * 0.1)
            assert ((m1[i].double().cpu() - rm).abs() <= 5 * 2.0 ** -24 * size + 1e-37).all()
            near(v1[i], rv, 6, "v")
            move = (rp - before[i].double().cpu() * (1 - HP["lr"] * HP["weight_decay"])).abs()
            size = before[i].double().abs().cpu() * 4 + move * 40 + HP["lr"] * 5 * (m0[i].double().abs().cpu() + 0.1) / (rv.sqrt() + 1e-8)
            assert ((p.double().cpu() - rp).abs() <= 2.0 ** -24 * size + 1e-37).all(), (name, i, step)
            if copy:
                assert torch.equal(copies[i], p.to(BF16))
    assert opt.state["step"] == 5


def test_matches_torch_in_structure(dev):
    """The same trajectory as the float64 recurrence over 30 steps of a quadratic."""
    say("adamw trajectory")
    target = torch.randn(700, generator=torch.Generator().manual_seed(3)).to(dev)
    p = torch.zeros(700, device=dev)
    ref, m, v = torch.zeros(700, dtype=torch.float64), torch.zeros(700, dtype=torch.float64), torch.zeros(700, dtype=torch.float64)
    opt = zs.AdamW([p], lr=0.05, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0)
    for t in range(1, 31):
        opt.step([p - target])
        ref, m, v = blockref.adamw(ref, ref - target.double().cpu(), m, v, 0.05, 0.9, 0.999, 1e-8, 0.0, t)
    # a step moves an entry by at most about lr; each of 30 steps repeats errors of a few ulps of it
    assert (p.double().cpu() - ref).abs().max() <= 30 * 0.05 * 100 * 2.0 ** -24


def code_values(opt):
    s = opt.state
    blocks = opt.total // 256
    mc, vc = s["m_code"].cpu(), s["v_code"].cpu()
    m = blockref.decode(mc & 127, 127, 8).view(blocks, 256) * s["m_scale"].double().cpu()[:, None]
    m = torch.where((mc >= 128).view(blocks, 256), -m, m).reshape(-1)
    r = (blockref.decode(vc, 255, 16).view(blocks, 256) * s["v_scale"].double().cpu()[:, None]).reshape(-1)
    return m, r


@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("copy", [False, True])
def test_8_bit_steps(dev, name, copy):
    """After each of four steps: parameters follow the step from the decoded moments; the new codes are one of the two
    neighbours of the exact value, zero only below the smallest code (and never for v > 0); scales are the blocks'
    largest magnitudes; padding stays zero."""
    sizes = SETS[name]
    say("adamw 8", name, copy)
    params = tensors(sizes, 1, dev)
    copies = [torch.full_like(p, 9, dtype=BF16) for p in params] if copy else None
    opt = zs.AdamW(params, copies=copies, state_bits=8, seed=77, **HP)
    if opt.total == 0:
        return
    live = torch.zeros(opt.total, dtype=torch.bool)
    for o, p in zip(opt.offsets, params):
        live[o:o + p.numel()] = True
    for step in range(1, 5):
        grads = tensors(sizes, 200 + step, dev, BF16 if copy else F32, 0.1)
        before = [p.clone() for p in params]
        m0, r0 = code_values(opt)
        opt.step(grads)
        flat = lambda ts: torch.cat([torch.cat([t.double().cpu(), torch.zeros(-t.numel() % 256, dtype=torch.float64)]) for t in ts])  # noqa: E731
        rp, rm, rv = blockref.adamw(flat(before), flat(grads), m0, r0 * r0, HP["lr"], *HP["betas"], HP["eps"], HP["weight_decay"], step)
        root = rv.sqrt()
        # moments from 8-bit values are exact to fp32 roundings, so the parameters are too
        move = (rp - flat(before) * (1 - HP["lr"] * HP["weight_decay"])).abs()
        size = flat(before).abs() * 4 + move * 60 + HP["lr"] * 5 * (m0.abs() + 0.1) / (root + 1e-8)
        assert ((flat(params) - rp).abs() <= 2.0 ** -24 * size + 1e-37)[live].all(), (name, step)
        if copy:
            assert all(torch.equal(a, b.to(BF16)) for a, b in zip(copies, params))
        m1, r1 = code_values(opt)
        ms, vs = opt.state["m_scale"].double().cpu(), opt.state["v_scale"].double().cpu()
        tol = 16 * 2.0 ** -24
        top_m, top_r = rm.abs().view(-1, 256).amax(1), root.view(-1, 256).amax(1)
        assert ((ms - top_m).abs() <= tol * top_m + 1e-30).all() and ((vs - top_r).abs() <= tol * top_r).all()
        # one code step around a value is at most 1/8 (m) or 1/16 (sqrt v) of it
        low_m, low_r = ms.repeat_interleave(256) * 2.0 ** -15, vs.repeat_interleave(256) * 2.0 ** -15
        assert ((m1 - rm).abs() <= rm.abs() * (1 / 8 + 1e-5) + low_m)[live].all()
        assert ((r1 - root).abs() <= root * (1 / 16 + 1e-5) + low_r)[live].all()
        assert (r1[live & (root > 0)] > 0).all()
        assert (m1[~live] == 0).all() and (r1[~live] == 0).all()
        dm, dv = opt.moments()
        assert torch.equal(dm.double().cpu(), m1.float().double()) or ((dm.double().cpu() - m1).abs() <= 2.0 ** -23 * m1.abs()).all()
        assert ((dv.double().cpu() - r1 * r1).abs() <= 2.0 ** -22 * r1 * r1 + 1e-37).all()


def test_8_bit_rounding_is_unbiased(dev):
    """A moment decaying by 0.1 % a step (beta2 = 0.999, zero gradients, one element holding the scale) follows its
    decay on average although a code step is 6 %."""
    say("adamw 8 drift")
    n = 256 * 400
    p = torch.zeros(n, device=dev)
    opt = zs.AdamW([p], lr=0.0, betas=(0.9, 0.999), state_bits=8, seed=5, weight_decay=0.0)
    first = torch.full((n,), 1.0, device=dev)
    first[::256] = 4.0
    opt.step([first])
    keep = torch.zeros(n, device=dev)
    start = opt.moments()[1].clone()
    for _ in range(200):
        keep[::256] = (opt.moments()[1][::256]).sqrt()   # holds the block's scale: v stays where it is
        opt.step([keep])
    v = opt.moments()[1]
    small = torch.ones(n, dtype=torch.bool, device=dev)
    small[::256] = False
    ratio = (v[small].sqrt().double().mean() / start[small].sqrt().double().mean()).item()
    # sqrt(0.999)^200 = 0.9048; an unbiased walk of 200 steps with a step of at most 1/16 has a spread below
    # sqrt(200) / 32 = 0.44 of an element, over 102000 elements 0.0014 of the mean: five times that
    assert abs(ratio - 0.999 ** 100) <= 0.007 * 0.999 ** 100 + 0.001


def test_padding_between_slices_and_guards(dev):
    """Parameters inside a larger buffer, at unaligned starts: neighbours keep their values; so do state elements
    behind a slice with 32-bit moments."""
    say("adamw guards")
    buf = torch.full((5000,), 3.0, device=dev)
    params = [buf[1:1 + 777], buf[1000:1000 + 1023], buf[3001:3001 + 5]]
    grads = [g.clone() for g in tensors([777, 1023, 5], 4, dev)]
    opt = zs.AdamW(params, **HP)
    for f in ("m", "v"):
        opt.state[f].fill_(0.5)
    opt.step(grads)
    mask = torch.ones(5000, dtype=torch.bool, device=dev)
    mask[1:778], mask[1000:2023], mask[3001:3006] = False, False, False
    assert (buf[mask] == 3).all() and (buf[~mask] != 3).any()
    for f in ("m", "v"):
        assert (opt.state[f][777:1024 - 0][:768 - 777 + 256] == 0.5).all()
    shifted = [torch.empty(n + 1, device=dev)[1:] for n in (777, 1023, 5)]
    for s, g in zip(shifted, grads):
        s.copy_(g)
    again = [torch.full((n,), 3.0, device=dev) for n in (777, 1023, 5)]
    other = zs.AdamW(again, **HP)
    for f in ("m", "v"):
        other.state[f].fill_(0.5)
    other.step(shifted)
    assert all(torch.equal(a, b) for a, b in zip(again, params))


@pytest.mark.parametrize("bits", [32, 8])
def test_missing_gradients_zero_and_non_finite(dev, bits):
    say("adamw special", bits)
    params = tensors([300, 300, 300, 300], 6, dev)
    opt = zs.AdamW(params, state_bits=bits, **HP)
    opt.step(tensors([300] * 4, 7, dev))
    before = [p.clone() for p in params]
    m0 = [t.clone() for t in slices(opt, opt.moments()[0])]
    g = tensors([300] * 4, 8, dev)
    g[1] = None
    g[2] = torch.zeros(300, device=dev)
    g[3][7], g[3][290] = float("nan"), float("inf")
    opt.step(g)
    m1 = slices(opt, opt.moments()[0])
    assert torch.equal(params[1], before[1]) and torch.equal(m1[1], m0[1])
    assert torch.isfinite(params[0]).all() and torch.isfinite(params[2]).all()
    assert torch.isnan(params[3][7]) and torch.isfinite(params[3][:7]).all()
    if bits == 8:   # a block with a value that is no number decodes to NaN, the next block is its own
        assert torch.isnan(m1[3][:256]).all()
    else:
        assert torch.isnan(m1[3][7]) and torch.isfinite(m1[3][:7]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_past_32_bits(dev, bits):
    """A tensor of more than 2^31 elements, and one behind it: the last elements move as those of a small tensor do."""
    say("adamw wide", bits)
    n = (1 << 31) + 1000
    tail = torch.randn(5000, generator=torch.Generator().manual_seed(2)).to(dev)
    p = torch.zeros(n, device=dev)
    g = torch.zeros(n, dtype=BF16, device=dev)
    p[-5000:], g[-5000:] = tail, 0.1 * tail.flip(0)
    q, h = tail.clone(), (0.1 * tail.flip(0)).to(BF16)
    opt = zs.AdamW([p, q], state_bits=bits, **HP)
    opt.step([g, h])
    small = zs.AdamW([tail.clone()], state_bits=bits, **HP)
    small.step([h])
    # from zero moments the parameters do not depend on how the moments are held
    assert torch.equal(p[-5000:], small.params[0]) and torch.equal(q, small.params[0])
    assert (p[:-5000] == 0).all()


def test_state_is_taken_over_and_graph(dev):
    say("adamw state, graph")
    for bits in (32, 8):
        a, b = tensors([1000, 33], 1, dev), tensors([1000, 33], 1, dev)
        x = zs.AdamW(a, state_bits=bits, seed=3, **HP)
        x.step(tensors([1000, 33], 2, dev))
        saved = {k: v.clone() if torch.is_tensor(v) else v for k, v in x.state.items()}
        for p, q in zip(a, b):
            q.copy_(p)
        y = zs.AdamW(b, state_bits=bits, state=saved, **HP)
        g = tensors([1000, 33], 3, dev)
        x.step(g)
        y.step(g)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert all(torch.equal(p, q) for p, q in zip(x.moments(), y.moments()))
        # capture: every replay is the step of the captured number on the current values
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            x.step(g)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            y.state["step"] = x.state["step"] - 1
            y.step(g)
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals(dev):
    say("refusals")
    p = torch.zeros(10, device=dev)
    for bad in ([], [p.cpu()], [p.view(2, 5).t()], [p, p], [p, p[5:]]):
        with pytest.raises(ValueError):
            zs.AdamW(bad)
    with pytest.raises(TypeError):
        zs.AdamW([p.bfloat16()])
    with pytest.raises(ValueError):
        zs.AdamW([p], state_bits=16)
    with pytest.raises(ValueError):
        zs.AdamW([p], copies=[])
    with pytest.raises(TypeError):
        zs.AdamW([p], copies=[torch.zeros(10, device=dev)])
    opt = zs.AdamW([p])
    for bad in ([], [torch.zeros(9, device=dev)], [torch.zeros(10)], [torch.zeros(20, device=dev)[::2]]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(TypeError):
        opt.step([torch.zeros(10, device=dev, dtype=torch.float64)])
    for name, value in (("lr", -1.0), ("lr", float("nan")), ("betas", (1.0, 0.9)), ("betas", (0.9, -0.1)), ("eps", -1e-8), ("weight_decay", -1.0)):
        o = zs.AdamW([torch.zeros(4, device=dev)])
        setattr(o, name, value)
        with pytest.raises(zs.ZsError):
            o.step([torch.ones(4, device=dev)])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("which", ["params", "copies"])
def test_memory_replaced_behind_the_optimizer(dev, bits, which):
    """Parameters and copies whose memory was replaced by one of another type, size, device or layout after the
    constructor looked at them are refused before any launch; one that fits is stepped."""
    say("replaced memory", bits, which)

    def make():
        params = [torch.nn.Parameter(torch.ones(600, device=dev)) for _ in range(3)]
        copies = [torch.zeros(600, dtype=BF16, device=dev) for _ in range(3)]
        return params, copies, zs.AdamW(params, copies=copies, state_bits=bits, **HP)
    kind = F32 if which == "params" else BF16
    other = BF16 if which == "params" else F32
    for bad, error in ((torch.zeros(600, dtype=other, device=dev), TypeError), (torch.zeros(300, dtype=kind, device=dev), ValueError),
                       (torch.zeros(0, dtype=kind, device=dev), ValueError), (torch.zeros(600, dtype=kind), ValueError),
                       (torch.zeros(1200, dtype=kind, device=dev)[::2], ValueError), (torch.zeros(600, dtype=torch.float64, device=dev), TypeError),
                       (torch.zeros(600, dtype=torch.float16, device=dev), TypeError)):
        params, copies, opt = make()
        (params if which == "params" else copies)[1].data = bad
        for grads in ([torch.ones(600, device=dev)] * 3, [torch.ones(600, device=dev), None, None]):
            with pytest.raises(error):
                opt.step(grads)
        assert opt.state["step"] == 0 and (params[0] == 1).all() and (copies[0] == 0).all() and (opt.moments()[0] == 0).all()
    module = torch.nn.Linear(20, 30, device=dev)   # as a model that is cast keeps its Parameters
    opt = zs.AdamW(module.parameters(), state_bits=bits, **HP)
    module.bfloat16()
    module(torch.ones(2, 20, dtype=BF16, device=dev)).sum().backward()
    with pytest.raises(TypeError):
        opt.step()
    params, copies, opt = make()
    (params if which == "params" else copies)[1].data = torch.ones(600, dtype=kind, device=dev)
    opt.step([torch.ones(600, device=dev)] * 3)
    assert torch.equal(params[1], params[0]) and torch.equal(copies[1], copies[0]) and (params[1] != 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_memory_shared_after_construction(dev, bits):
    """Parameters and copies that share memory since the constructor looked at them are refused; ones that merely moved
    are stepped where they are now."""
    say("shared memory", bits)
    one = [torch.ones(600, device=dev)] * 3
    for move in (lambda p, c: setattr(p[1], "data", p[0].data), lambda p, c: setattr(c[2], "data", c[0].data),
                 lambda p, c: setattr(c[1], "data", p[1].data.view(BF16)[:600]),
                 lambda p, c: setattr(p[2], "data", torch.cat([p[0].data, p[1].data])[:600]) or setattr(p[1], "data", p[2].data)):
        params, copies = [torch.ones(600, device=dev) for _ in range(3)], [torch.zeros(600, dtype=BF16, device=dev) for _ in range(3)]
        opt = zs.AdamW(params, copies=copies, state_bits=bits, **HP)
        opt.step(one)
        before = [t.clone() for t in (*params, *opt.moments())]
        move(params, copies)
        with pytest.raises(ValueError, match="share memory"):
            opt.step(one)
        with pytest.raises(ValueError, match="share memory"):
            opt.step(one)
        assert opt.state["step"] == 1 and torch.equal(params[0], before[0]) and torch.equal(opt.moments()[0], before[3])
    params, copies = [torch.ones(600, device=dev) for _ in range(3)], [torch.zeros(600, dtype=BF16, device=dev) for _ in range(3)]
    opt = zs.AdamW(params, copies=copies, state_bits=bits, **HP)
    old = params[0].data
    params[0].data, params[1].data = params[1].data, params[0].data.clone()
    opt.step(one)
    assert (old == 1).all() and torch.equal(params[0], params[2]) and torch.equal(params[1], params[2]) and (params[2] != 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_state_replaced_behind_the_optimizer(dev, bits):
    """State arrays put into the dictionary in place of the first ones: refused unless they have their type, size,
    device and layout; those that do are the state from then on."""
    say("replaced state", bits)
    for name in ("m", "v") if bits == 32 else ("m_code", "m_scale", "v_code", "v_scale"):
        p = torch.ones(600, device=dev)
        opt = zs.AdamW([p], state_bits=bits, **HP)
        old = opt.state[name]
        for bad, error in ((old[:-1].clone(), ValueError), (old.cpu(), ValueError), (old.double(), TypeError), (old.repeat(2)[::2], ValueError), (None, ValueError),
                           (old.view(1, -1), ValueError)):
            opt.state[name] = bad
            with pytest.raises(error):
                opt.step([torch.ones(600, device=dev)])
            if bits == 8:   # 32-bit moments are handed back as they are
                with pytest.raises(error):
                    opt.moments()
        opt.state[name] = old.clone()
        opt.step([torch.ones(600, device=dev)])
        assert opt.state["step"] == 1 and (p != 1).all() and (old == 0).all() and (opt.state[name] != 0).any()


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_count_as_changes(dev, bits):
    """A step counts as a change of the parameters and copies it writes: a graph built before it refuses its backward,
    as after any change in place.  A parameter without a gradient is not written and does not count."""
    say("versions", bits)
    p, q = (torch.randn(40, device=dev).requires_grad_() for _ in range(2))
    copies = [torch.zeros(40, dtype=BF16, device=dev) for _ in range(2)]
    opt = zs.AdamW([p, q], copies=copies, state_bits=bits, **HP)
    loss = (p * p).sum()
    other = (q * q).sum()
    seen = [t._version for t in (p, q, *copies)]
    opt.step([torch.ones(40, device=dev), None])
    assert [t._version > v for t, v in zip((p, q, *copies), seen)] == [True, False, True, False]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    other.backward()
    opt.step([torch.ones(40, device=dev), q.grad])
    assert q._version > seen[1] and copies[1]._version > seen[3]
