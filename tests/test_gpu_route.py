"""Routing to experts and its gradient against float64, the choice against the definition row by row, on the GPU."""
import math

import pytest
import torch

import edge_node_scatter_amd as zs
import layersref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = math.inf


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.load()
    return torch.device("cuda:0")


def say(*a):
    print("[gpu]", *a, flush=True)


def check(x, router, bias, dev, gw_seed=0, what=""):
    """Choice, weights and gradients of one call."""
    xd, bd = x.to(dev), None if bias is None else bias.to(dev)
    weight, expert = zs.zs_route(xd, router, bd)
    w_ref, e_ref = ref.route(x, router, bias)
    assert torch.equal(expert.cpu(), e_ref), (what, (expert.cpu() != e_ref).nonzero()[:3])
    # formed in 64 bits, rounded to fp32 once.  Only a softmax's sum over all experts is one of fp32 exponentials: each
    # is off by an ulp (2 half ulps) and by |d| half ulps for the rounding of its argument d = x - max; on average over
    # the terms' sizes |d| is at most the logarithm of their number (the terms' entropy), below 7 for 1024.
    sums = 9 * 2.0 ** -24 if router.score == "softmax" and not router.renormalise else 0.0
    got = weight.double().cpu()
    assert torch.equal(got.isnan(), w_ref.isnan()), what
    ok = ((got - w_ref).abs() <= (2.0 ** -24 + 1e-12 + sums) * w_ref.abs() + 1e-44) | w_ref.isnan()
    assert bool(ok.all()), what
    gw = torch.randn(expert.shape, generator=torch.Generator().manual_seed(gw_seed))
    gx = zs.zs_route_backward(gw.to(dev), xd, expert, router).double().cpu()
    g_ref, bound = ref.route_grad(gw, x, e_ref, router)
    ok = ((gx - g_ref).abs() <= bound(x.dtype)) | (gx.isnan() & g_ref.isnan())
    assert bool(ok.all()), (what, ((gx - g_ref).abs() - bound(x.dtype)).max().item())
    return weight, expert, gx


EXPERTS = [(1, 1), (2, 1), (5, 2), (8, 2), (9, 9), (16, 4), (31, 3), (32, 32), (33, 5), (64, 6), (65, 8), (128, 2), (130, 64), (256, 8), (257, 4), (500, 10), (512, 1), (777, 16), (1024, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,k", EXPERTS)
def test_route(dev, dtype, score, n, k):
    g = torch.Generator().manual_seed(n + k)
    for M in (1, 37):
        x = (2 * torch.randn(M, n, generator=g)).to(dtype)
        bias = 0.1 * torch.randn(n, generator=g)
        for renorm in (True, False):
            say("route", dtype, score, M, n, k, renorm)
            r = zs.Router(n, k, score=score, renormalise=renorm, scale=2.5)
            check(x, r, None, dev, what="plain")
            check(x, r, bias, dev, what="bias")
            check(x, r, torch.zeros(n), dev, what="no bias yet")   # with bf16's many equal logits


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups,top,k", [(8, 2, 1, 2), (8, 8, 3, 3), (16, 4, 2, 4), (60, 3, 2, 7), (64, 64, 5, 5), (160, 8, 3, 6), (256, 8, 4, 8), (255, 5, 2, 8), (512, 16, 1, 8), (1024, 64, 7, 20), (1000, 8, 8, 64)])
def test_route_groups(dev, score, n, groups, top, k):
    g = torch.Generator().manual_seed(n)
    for dtype in (F32, BF16):
        x = (2 * torch.randn(40, n, generator=g)).to(dtype)
        bias = 0.1 * torch.randn(n, generator=g)
        for best in (1, 2):
            say("groups", dtype, score, n, groups, top, k, best)
            r = zs.Router(n, k, score=score, groups=groups, top_groups=top, best=best, renormalise=best == 2)
            check(x, r, bias, dev, what="bias")
            check(x, r, None, dev, what="no bias")
            check(x, r, torch.zeros(n), dev, what="no bias yet")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_experts(dev, dtype, score):
    """Experts switched off by -inf or the type's lowest value, rows with few or none left, through logits and bias."""
    g = torch.Generator().manual_seed(3)
    low = torch.finfo(dtype).min
    for n, groups, k in ((12, 1, 4), (64, 8, 5), (300, 1, 8), (300, 10, 8)):
        say("masked", dtype, score, n, groups)
        x = torch.randn(60, n, generator=g).to(dtype)
        x[torch.rand(60, n, generator=g) < 0.5] = -INF
        x[5:10] = -INF
        x[10:15] = low
        x[15:20, 1:] = -INF
        x[20:25][torch.rand(5, n, generator=g) < 0.7] = low
        x[25:30, :-2] = -INF
        x[30, :] = -INF
        x[30, n // 2] = low
        bias = 0.2 * torch.randn(n, generator=g)
        bias[1], bias[3] = -INF, math.nan
        bias[n - 1] = INF if score == "sigmoid" else 3.0
        for renorm in (True, False):
            r = zs.Router(n, k, score=score, groups=groups, top_groups=max(1, groups // 2), renormalise=renorm)
            for b in (None, bias):
                weight, expert, gx = check(x, r, b, dev, what=(n, groups, renorm, b is None))
                assert (expert[5:10] == n).all() and (weight[5:10] == 0).all() and (gx[5:10] == 0).all()
            r = zs.Router(n, k, score=score, groups=groups, top_groups=groups, renormalise=renorm)
            check(x, r, torch.full((n,), -INF), dev, what="all off by bias")


def test_rows_that_are_not_numbers(dev):
    say("nan rows")
    g = torch.Generator().manual_seed(4)
    for n in (8, 40, 256):
        x = torch.randn(30, n, generator=g)
        x[3, 5] = math.nan
        x[4, 0] = INF
        x[6] = math.nan
        for score in ("softmax", "sigmoid"):
            for bias in (None, torch.zeros(n)):
                r = zs.Router(n, 3, score=score, groups=4, top_groups=2)
                weight, expert = zs.zs_route(x.to(dev), r, None if bias is None else bias.to(dev))
                rows = [3, 6] + ([4] if score == "softmax" else [])
                assert weight[rows].isnan().all() and (expert[rows] == n).all()
                fine = [i for i in range(30) if i not in rows]
                w_ref, e_ref = ref.route(x[fine], r, bias)
                assert torch.equal(expert[fine].cpu(), e_ref) and not weight[fine].isnan().any()


def test_ties_go_to_the_lowest_index(dev):
    say("ties")
    for n in (8, 20, 64, 100, 256, 512, 1000):
        x = torch.zeros(3, n)
        x[1, n // 2:] = 1.0
        for r in (zs.Router(n, min(n // 2, 8)), zs.Router(n, min(n // 4, 8), groups=4, top_groups=2), zs.Router(n, 2, score="sigmoid", groups=4, top_groups=1)):
            for bias in (None, torch.zeros(n)):
                _, expert = zs.zs_route(x.to(dev), r, None if bias is None else bias.to(dev))
                first = torch.arange(r.k)
                assert torch.equal(expert.cpu(), torch.stack([first, first + n // 2, first]))


def test_close_scores(dev):
    """Experts whose scores differ by less than fp32 holds: the order is that of 64 bits."""
    say("close scores")
    g = torch.Generator().manual_seed(6)
    for n, groups in ((16, 1), (64, 1), (256, 8), (256, 1)):
        for score in ("softmax", "sigmoid"):
            # logits of a few neighbouring fp32 values, biases that nearly undo them
            x = 1.0 + torch.randint(0, 4, (200, n), generator=g) * 2.0 ** -23
            bias = -(torch.randint(0, 4, (n,), generator=g) * 2.0 ** -26)
            r = zs.Router(n, 6, score=score, groups=groups, top_groups=max(1, groups // 2))
            check(x, r, bias, dev, what=(n, score))
            check(x, r, None, dev, what=(n, score))
            # saturated scores
            x = 20 + 4 * torch.randn(200, n, generator=g)
            check(x, zs.Router(n, 6, score=score, renormalise=False), 1e-9 * torch.randn(n, generator=g), dev, what="saturated")
            # scores far below 1 with a bias that chooses them
            x = -90 + 8 * torch.randn(200, n, generator=g)
            x[:, 0] = 3.0
            check(x, zs.Router(n, 4, score=score), torch.randn(n, generator=g), dev, what="small")
            check(8 * x, zs.Router(n, 4, score=score), torch.randn(n, generator=g), dev, what="no score in 64 bits")


def test_many_rows(dev):
    """More rows than a round of workgroups, against the same calls on parts (which the tests above hold to the definition)."""
    say("many rows")
    g = torch.Generator().manual_seed(7)
    for M, n, groups, k, dtype in ((70001, 256, 8, 8, BF16), (33333, 8, 1, 2, F32), (20011, 160, 1, 6, F32)):
        x = torch.randn(M, n, generator=g).to(dtype).to(dev)
        bias = 0.1 * torch.randn(n, generator=g).to(dev)
        r = zs.Router(n, k, score="sigmoid", groups=groups, top_groups=(groups + 1) // 2)
        weight, expert = zs.zs_route(x, r, bias)
        gw = torch.randn(M, k, device=dev)
        gx = zs.zs_route_backward(gw, x, expert, r)
        for at in (slice(0, 50), slice(M // 2, M // 2 + 50), slice(M - 50, M)):
            w2, e2 = zs.zs_route(x[at], r, bias)
            assert torch.equal(weight[at], w2) and torch.equal(expert[at], e2)
            assert torch.equal(gx[at], zs.zs_route_backward(gw[at], x[at], e2, r))
        assert (expert >= 0).all() and (expert < n).all()
        w_ref, e_ref = ref.route(x[-200:].cpu(), r, bias.cpu())
        assert torch.equal(expert[-200:].cpu(), e_ref)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups,k", [(256, 8, 8), (128, 1, 6), (60, 4, 4), (512, 16, 10), (1024, 1, 12), (16, 1, 2)])
def test_choice_over_many_rows(dev, score, n, groups, k):
    """Every choice of 40000 rows, among them rows that fp32 sums cannot tell, against stable sorts in float64."""
    say("many choices", score, n, groups, k)
    g = torch.Generator().manual_seed(n + k)
    M = 40000
    top = max(1, groups // 2)
    for dtype, spread in ((F32, 1.5), (BF16, 1.5), (F32, 1e-3), (F32, 1e-6)):
        x = (spread * torch.randn(M, n, generator=g)).to(dtype).to(dev)
        bias = (0.3 * spread * torch.randn(n, generator=g)).to(dev)
        _, expert = zs.zs_route(x, zs.Router(n, k, score=score, groups=groups, top_groups=top), bias)
        s = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), 1)
        q = s + bias.double()
        if groups > 1:
            best = q.view(M, groups, -1).sort(2, descending=True)[0][:, :, :2].sum(2)
            order = best.sort(dim=1, descending=True, stable=True)[1][:, :top]
            stay = torch.zeros(M, groups, dtype=torch.bool, device=dev).scatter_(1, order, True)
            q = q.masked_fill(~stay.repeat_interleave(n // groups, 1), -INF)
        ref_q, ref_e = q.sort(dim=1, descending=True, stable=True)
        # rows whose order hangs on the last bits of float64 (a softmax's sum in another order) are left out
        gap = (ref_q[:, :k] - ref_q[:, 1:k + 1] if n > k else ref_q[:, :k - 1] - ref_q[:, 1:k]).amin(1)
        sure = gap > 1e-14
        if groups > 1:
            sure &= (lambda b: b[:, top - 1] - b[:, top])(best.sort(1, descending=True)[0]) > 1e-14
        assert sure.float().mean() > 0.9
        assert torch.equal(expert[sure], ref_e[sure][:, :k]), (dtype, spread)


def test_layouts(dev):
    say("layouts")
    g = torch.Generator().manual_seed(8)
    big = torch.randn(200, 200, generator=g).to(dev)
    r = zs.Router(64, 4, score="softmax", renormalise=False)
    for x in (big[:50, :64], big[3:53, 5:69], big.T[:50, :64], big[:1, :64].expand(50, 64)):
        w, e = zs.zs_route(x, r)
        w2, e2 = zs.zs_route(x.contiguous(), r)
        assert torch.equal(w, w2) and torch.equal(e, e2)
        gw = torch.randn(4, 50, generator=g).to(dev).T   # another order of strides
        assert torch.equal(zs.zs_route_backward(gw, x, e, r), zs.zs_route_backward(gw.contiguous(), x.contiguous(), e, r))
    bias = torch.randn(200, generator=g).to(dev)
    w, e = zs.zs_route(big[:50, :64], r, bias[1:65])
    w2, e2 = zs.zs_route(big[:50, :64], r, bias[1:65].clone())
    assert torch.equal(w, w2) and torch.equal(e, e2)
    out = zs.zs_route(big[:0, :64], r)
    assert out[0].shape == (0, 4) and out[1].shape == (0, 4)


def test_backward_of_any_choice(dev):
    """Slots outside the experts have no part; one expert in two slots gets both slots' gradients."""
    say("any choice")
    g = torch.Generator().manual_seed(9)
    for n in (8, 50, 300):
        x = torch.randn(40, n, generator=g)
        expert = torch.randint(0, n, (40, 5), generator=g)
        expert[3], expert[4, 2], expert[5, 0], expert[6] = n, -1, 1 << 40, 2
        gw = torch.randn(40, 5, generator=g)
        gw[4, 2] = math.nan   # of a slot that holds nothing
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                r = zs.Router(n, 5, score=score, renormalise=renorm, scale=0.5)
                got = zs.zs_route_backward(gw.to(dev), x.to(dev), expert.to(dev), r).double().cpu()
                want, bound = ref.route_grad(torch.nan_to_num(gw, nan=0.0), x, expert, r)
                assert ((got - want).abs() <= 4 * bound(F32) + 1e-7).all(), (n, score, renorm)


def test_gradient_against_differences(dev):
    say("differences")
    g = torch.Generator().manual_seed(10)
    x, c = torch.randn(20, 24, generator=g).to(dev), torch.randn(20, 4, generator=g).to(dev)
    d = torch.randn(20, 24, generator=g).to(dev)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            r = zs.Router(24, 4, score=score, renormalise=renorm)
            _, expert = zs.zs_route(x, r)
            h, keep = 2.0 ** -10, []
            lo, hi = zs.zs_route(x - h * d, r), zs.zs_route(x + h * d, r)
            keep = (lo[1] == expert).all(1) & (hi[1] == expert).all(1)   # rows whose choice is the same on both sides
            assert keep.sum() >= 15
            gx = torch.autograd.grad((zs.route(x.requires_grad_(), r)[0] * c).sum(), x)[0]
            x = x.detach()
            slope = ((hi[0] - lo[0]).double() * c).sum(1) / (2 * h)
            exact = (gx * d).double().sum(1)
            # h^2 of a third derivative of order |d|^3 <= 50, and 2^-24 / h for each of four weights of order one
            assert ((slope - exact).abs() <= 50 * h * h + 8 * 2.0 ** -24 / h * c.abs().amax(1))[keep].all()


def test_graph_and_stream(dev):
    say("graph")
    g = torch.Generator().manual_seed(12)
    x, bias = torch.randn(700, 160, generator=g).to(dev), 0.1 * torch.randn(160, generator=g).to(dev)
    gw = torch.randn(700, 6, generator=g).to(dev)
    r = zs.Router(160, 6, score="sigmoid", groups=8, top_groups=3)

    def run():
        w, e = zs.zs_route(x, r, bias)
        groups = zs.expert_groups(e, 160)
        return w, e, zs.zs_route_backward(gw, x, e, r), groups.rowptr, groups.perm
    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run()
    for i in range(4):
        x.copy_(x.roll(1, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(), res)), i


def test_refusals(dev):
    say("refusals")
    r = zs.Router(16, 2)
    x, e, w = torch.zeros(5, 16, device=dev), torch.zeros(5, 2, dtype=torch.int64, device=dev), torch.zeros(5, 2, device=dev)
    for call in (lambda: zs.zs_route(x[:, :8], r), lambda: zs.zs_route(x[0], r), lambda: zs.zs_route(x, r, torch.zeros(8, device=dev)), lambda: zs.zs_route(x, r, torch.zeros(16)),
                 lambda: zs.zs_route_backward(w[:4], x, e, r), lambda: zs.zs_route_backward(w, x, e[:, :1], r), lambda: zs.zs_route_backward(w, x, e.cpu(), r), lambda: zs.expert_groups(e[:, 0], 16)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: zs.zs_route(x.half(), r), lambda: zs.zs_route(x, r, torch.zeros(16, device=dev).bfloat16()), lambda: zs.zs_route_backward(w.bfloat16(), x, e, r),
                 lambda: zs.zs_route_backward(w, x, e.int(), r), lambda: zs.expert_groups(e.int(), 16)):
        with pytest.raises(TypeError):
            call()


def test_experts_groups(dev):
    """Slots without an expert are rows of no group: their products are zeros."""
    say("expert groups")
    g = torch.Generator().manual_seed(14)
    x = torch.randn(40, 6, generator=g)
    x[7] = -INF
    x[9, 1:] = -INF
    r = zs.Router(6, 3)
    w, e = zs.zs_route(x.to(dev), r)
    groups = zs.expert_groups(e, 6)
    flat = e.cpu().reshape(-1)
    live = flat < 6
    assert torch.equal(groups.rowptr.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat[live], minlength=6).cumsum(0)]))
    rows, mats = torch.randn(120, 8, generator=g), torch.randn(6, 8, 4, generator=g)
    y = zs.zs_grouped_mm(rows.to(dev), mats.to(dev), groups).cpu()
    assert (y[~live] == 0).all() and (~live).sum() == 5
    assert torch.allclose(y[live], torch.bmm(rows[live][:, None], mats[flat[live]])[:, 0], atol=1e-5)
