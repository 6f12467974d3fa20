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
