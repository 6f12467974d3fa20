"""Routing where fp32 is at its limits: biases that are no numbers or the type's lowest, confident rows, rows beside rows
that have to be settled in fp64.  Against float64, on the GPU."""
import math

import pytest
import torch

import edge_node_scatter_amd as zs
import layersref as ref
from test_gpu_route import check, dev, say  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = math.inf
LOW = torch.finfo(F32).min
GROUPED = [(16, 2, 1), (16, 4, 2), (60, 3, 1), (64, 8, 3), (160, 8, 3), (256, 8, 4), (255, 5, 2), (512, 16, 5), (1000, 8, 3), (1024, 64, 7)]


# ---- which groups stay --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_bias_that_is_no_number(dev, score):  # noqa: F811
    """Such an expert is not there: it has no part in its group's score, wherever in the group it stands."""
    for n, groups, top in GROUPED:
        say("NaN bias", score, n, groups)
        g = torch.Generator().manual_seed(n + groups)
        x, k = torch.randn(60, n, generator=g), min(4, n // groups)
        # one clear best expert in every group, the seconds decide; a third of the others is not there
        bias = 0.02 * torch.randn(n, generator=g) - 0.5
        lead = torch.arange(groups) * (n // groups) + torch.randint(0, max(1, n // groups // 2), (groups,), generator=g)
        off = torch.rand(n, generator=g) < 0.34
        off[lead] = False
        off[lead + 1] = True
        bias[lead] = 0.5 + 0.3 * torch.rand(groups, generator=g)
        bias[off] = math.nan
        for best in (1, 2):
            check(x, zs.Router(n, k, score=score, groups=groups, top_groups=top, best=best), bias, dev, what=(n, best))
    # the first group's best alone would win if it counted twice
    bias = torch.tensor([0.5, math.nan] + [-0.4] * 6 + [0.2] * 8)
    for dtype in (F32, BF16):
        _, expert, _ = check(torch.zeros(5, 16, dtype=dtype), zs.Router(16, 3, score=score, groups=2), bias, dev)
        assert (expert >= 8).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_whose_sums_leave_fp32(dev, score):  # noqa: F811
    """The type's lowest value as a mask, and biases whose sum is above its largest: experts that are there all the same."""
    for n, groups, top in GROUPED:
        say("large biases", score, n, groups)
        g = torch.Generator().manual_seed(n + groups)
        x, k, per = torch.randn(6, n, generator=g), min(4, n // groups), n // groups
        for best in (1, 2):
            for keep in (0, 1, top, groups):   # groups with ordinary biases; of the rest all or all but one expert is masked
                for left in (0, 1):
                    bias = torch.full((n,), LOW)
                    for i in torch.randperm(groups, generator=g)[:keep].tolist():
                        bias[i * per:(i + 1) * per] = 0.1 * torch.randn(per, generator=g)
                    if left:
                        bias[per - 1::per] = -0.3
                    for tops in {top, groups}:
                        _, expert, _ = check(x, zs.Router(n, k, score=score, groups=groups, top_groups=tops, best=best), bias, dev, what=(n, best, keep, left, tops))
                        assert (expert < n).all()
            # sums of two that are both beyond the type, far apart and equal
            bias = torch.where(torch.rand(n, generator=g) < 0.5, -1.0, 1.0) * (2.0 + 1.4 * torch.rand(n, generator=g)) * 1e38
            check(x, zs.Router(n, k, score=score, groups=groups, top_groups=top, best=best), bias, dev, what=(n, best, "random"))
            check(x, zs.Router(n, k, score=score, groups=groups, top_groups=top, best=best), bias.abs().clamp(min=3e38), dev, what=(n, best, "above"))


# ---- gradients of confident rows ----------------------------------------------------------------------------------

def scores64(x, sigmoid):
    return torch.sigmoid(x.double()) if sigmoid else torch.softmax(x.double(), 1)


def softmax_grad(gw, x, expert, scale):
    """Gradient of the logits from that of unnormalised softmax weights, and the size of its terms: with G_e the sum of
    the gradients of e's slots, dx_e = s_e sum over f of s_f (G_e - G_f), which has no difference of large terms."""
    s = scores64(x, False)
    G = torch.zeros_like(s).scatter_add_(1, expert, gw.double() * scale)
    d = G[:, :, None] - G[:, None, :]
    return s * (s[:, None, :] * d).sum(2), s * (s[:, None, :] * d.abs()).sum(2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_of_a_confident_softmax(dev, dtype):  # noqa: F811
    """One expert far ahead: its weight is nearly 1, its gradient the small rest of it."""
    for n, k in ((8, 1), (20, 1), (64, 1), (64, 3), (160, 6), (300, 2), (1000, 1), (1024, 16)):
        say("confident softmax", dtype, n, k)
        g = torch.Generator().manual_seed(n + k)
        x = torch.randn(48, n, generator=g)
        margin = torch.tensor([0.0, 4, 8, 10, 12, 14, 16, 18, 20, 25, 30, 36]).repeat(4)
        x[torch.arange(48), torch.randint(0, n, (48,), generator=g)] += 5 + margin
        x = x.to(dtype)
        r = zs.Router(n, k, renormalise=False, scale=1.5)
        _, expert = zs.zs_route(x.to(dev), r)
        gw = torch.randn(48, k, generator=g)
        if k > 2:   # a choice of the caller's own: an expert in two slots
            expert[::3, 2] = expert[::3, 0]
        got = zs.zs_route_backward(gw.to(dev), x.to(dev), expert, r).double().cpu()
        want, size = softmax_grad(gw, x, expert.cpu(), 1.5)
        # a score that is an fp32 exponential: two ulps (4 half ulps), the rounding of its argument d (|d| half ulps), the
        # rounding of the factors and the product 4; 88 and more below the largest it is 0
        d = (x.double() - x.double().amax(1, keepdim=True)).abs().amax(1, keepdim=True)
        bound = ref.rounded(want, (8 + 2 * d) * ref.HALF * size, dtype)
        over = ((got - want).abs() - bound).max().item()
        assert over <= 0, (n, k, over, ((got - want).abs() / bound).max().item())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_a_confident_share(dev, dtype, score):  # noqa: F811
    """Renormalised weights of which one is nearly 1."""
    for n, k in ((8, 2), (20, 3), (64, 6), (300, 2), (1024, 64)):
        say("confident share", dtype, score, n, k)
        g = torch.Generator().manual_seed(n + k)
        x = torch.randn(36, n, generator=g)
        margin = torch.tensor([0.0, 8, 12, 16, 20, 25, 30, 36, 40]).repeat(4)
        if score == "softmax":
            x[torch.arange(36), torch.randint(0, n, (36,), generator=g)] += margin
        else:   # (its scores differ by a factor only below 0)
            x -= margin[:, None]
            x[torch.arange(36), torch.randint(0, n, (36,), generator=g)] = 0.5
        x = x.to(dtype)
        r = zs.Router(n, k, score=score, scale=2.5)
        _, expert = zs.zs_route(x.to(dev), r)
        gw = torch.randn(36, k, generator=g)
        gw[::4] = gw[::4, :1]   # one gradient for all: nothing is left
        got = zs.zs_route_backward(gw.to(dev), x.to(dev), expert, r).double().cpu()
        e = expert.cpu()
        v = x.double().gather(1, e)
        p = torch.softmax(v if score == "softmax" else torch.nn.functional.logsigmoid(v), 1)
        rest = 1.0 if score == "softmax" else torch.sigmoid(-v)
        d = 2.5 * gw.double()
        d = d[:, :, None] - d[:, None, :]
        part, size = p * (p[:, None, :] * d).sum(2) * rest, p * (p[:, None, :] * d.abs()).sum(2) * rest
        want, size = (torch.zeros(36, n, dtype=torch.float64).scatter_(1, e, t) for t in (part, size))
        # fp64 throughout: 64 additions, some products and exponentials
        bound = ref.rounded(want, 256 * 2.0 ** -53 * size, dtype) + ref.HALF * want.abs()
        over = ((got - want).abs() - bound).max().item()
        assert over <= 0, (n, k, over, ((got - want).abs() / bound).max().item())


# ---- rows beside others -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("n,k", [(8, 2), (32, 4), (64, 6), (128, 8), (256, 8), (1000, 16)])
def test_a_row_is_the_same_beside_others(dev, n, k):  # noqa: F811
    """The bits of a row's weights do not depend on the rows that are computed with it, some of which have experts too
    close for fp32, and some more of them than there are candidates."""
    say("rows beside others", n, k)
    g = torch.Generator().manual_seed(n)
    M = 96
    x = 2 * torch.randn(M, n, generator=g)
    bias = 0.1 * torch.randn(n, generator=g)
    bias[:2] = 0.9   # among the chosen ones, equal
    x[::5, 1] = x[::5, 0] + 2.0 ** -22
    x[3::16] = 0.25 + 2.0 ** -23 * torch.randint(0, 2, (M // 16, n), generator=g)
    for score in ("softmax", "sigmoid"):
        for b in (bias, bias.clamp(max=0.9).round(decimals=1)):
            for renorm in (False, True):
                r = zs.Router(n, k, score=score, renormalise=renorm)
                weight, expert = zs.zs_route(x.to(dev), r, b.to(dev))
                for row in range(M):
                    w, e = zs.zs_route(x[row:row + 1].to(dev), r, b.to(dev))
                    assert torch.equal(expert[row:row + 1], e), row
                    assert torch.equal(weight[row:row + 1].view(torch.int32), w.view(torch.int32)), (score, renorm, row)
                check(x, r, b, dev, what=(score, renorm))
