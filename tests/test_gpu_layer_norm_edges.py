"""Layer norm of rows that lie far from zero for their spread, against float64, on the GPU."""
import pytest
import torch

import edge_node_scatter_amd as zs
import layersref as ref
from test_gpu_layers import BF16, F32, dev, mk, gen, say, within  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [3, 30, 61, 115, 257, 500, 777, 892, 899, 1000, 1021, 1031, 2000, 2047, 4100, 8191])
def test_constant_rows(dev, dtype, c):  # noqa: F811
    """Nothing deviates from the mean, whatever the sum's roundings: y is the bias, the gradients those of xh = 0."""
    say("constant rows", dtype, c)
    v = torch.tensor([0.0, 1e-30, 3.7, -123.456, 1.9e4, 1.1e6, -3.3e7, 7.3e9, 2.1e11, 1e12, -4.4e13, 3.3e15, 9.1e17, 1e20, -7e24, 1.3e30])
    x = v.to(dtype)[:, None].repeat(1, c)
    g = gen(c)
    w, b, gy = 1 + 0.2 * mk(g, c), mk(g, c), mk(g, len(v), c, dtype=dtype)
    # xh is within 64 half ulps of 0 (the reference's bound), as are the products with it
    y = zs.zs_layer_norm(x.to(dev), w.to(dev), b.to(dev))
    want = b.double().expand(len(v), c)
    within(y, want, ref.rounded(want, ref.HALF * (64 * w.double().abs() + 4 * b.double().abs()), dtype), "y")
    gx, gw, gb = zs.zs_layer_norm_backward(gy.to(dev), x.to(dev), w.to(dev))
    r, t = 1e-5 ** -0.5, gy.double() * w.double()
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    want = r * (t - mean(t))
    inner = 128 * ref.HALF * r * (t.abs() + 3 * mean(t.abs()))
    within(gx, want, ref.rounded(want, inner, dtype), "grad_x")
    within(gw, torch.zeros(c, dtype=torch.float64), 64 * ref.HALF * gy.double().abs().sum(0), "grad_w")


@pytest.mark.parametrize("c", [30, 257, 777, 892, 1024, 2000, 4100, 8191])
def test_spreads_of_few_ulps(dev, c):  # noqa: F811
    """Rows of a few neighbouring fp32 values, far from zero."""
    say("few ulps", c)
    g = gen(c)
    rows = []
    for at in (2.0 ** 10, 2.0 ** 20, 1.5 * 2.0 ** 24, 2.0 ** 30, 1.25 * 2.0 ** 40):
        ulp = torch.finfo(F32).eps * 2.0 ** torch.tensor(at).log2().floor()
        for spread in (1, 3, 30):
            rows.append(at + ulp * torch.randint(0, spread + 1, (c,), generator=g))
        rows.append(torch.full((c,), at))
        rows[-1][c // 2] += ulp   # one element beside the others
    x = torch.stack(rows).float()
    w, b, gy = 1 + 0.2 * mk(g, c), mk(g, c), mk(g, len(rows), c)
    # float64 sums of these are exact or off by 2^-53 of the mean, far below an ulp of fp32
    want, bound = ref.layer_norm(x, w, b, 1e-5)
    within(zs.zs_layer_norm(x.to(dev), w.to(dev), b.to(dev)), want, bound(F32), "y")
    (gx, gw, gb), (bx, bw, bb) = ref.layer_norm_grads(gy, x, w, 1e-5)
    got = zs.zs_layer_norm_backward(gy.to(dev), x.to(dev), w.to(dev))
    within(got[0], gx, bx(F32), "grad_x")
    within(got[1], gw, bw(), "grad_w")
    within(got[2], gb, bb(), "grad_b")
