"""Grouped products and their gradients against float64, through the binding on the GPU."""
import numpy as np
import pytest
import torch

import blockref
import edge_node_scatter_amd as zs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.load()
    return torch.device("cuda:0")


def say(*a):
    print("[gpu]", *a, flush=True)


def make(M, G, k, n, dtype, perm, seed, empty=True, outside=False):
    """x, w, grad_y, offsets, perm on the CPU; every third group empty, and rows outside all groups on request."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    share = rng.random(G) + 0.1
    if empty and G >= 3:
        share[1::3] = 0
    lo, hi = (M // 5, M - M // 7) if outside else (0, M)
    at = lo + np.concatenate([[0], np.round(np.cumsum(share) / share.sum() * (hi - lo))])
    offsets = torch.from_numpy(at.astype(np.int32))
    p = torch.from_numpy(rng.permutation(M).astype(np.int32)) if perm else None
    mk = lambda *s: torch.randn(*s, generator=gen).to(dtype)  # noqa: E731
    return mk(M, k), mk(G, k, n), mk(M, n), offsets, p


def groups_of(offsets, perm, dev):
    return zs.Csr(offsets.to(dev), None if perm is None else perm.to(dev), None, len(offsets) - 1)


def close(got, ref, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    worst = ((got - ref).abs() / bound).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"


SIZES = [(1, 1, 1, 1), (1, 3, 8, 8), (2, 5, 16, 33), (7, 2, 3, 5), (31, 1, 64, 17), (96, 4, 64, 64), (129, 4, 64, 128),
         (300, 9, 33, 47), (513, 16, 96, 32), (700, 3, 32, 96), (1000, 5, 130, 260), (257, 2, 520, 136), (2500, 70, 40, 24),
         (64, 2, 1024, 512), (5, 4, 1000, 1032), (3000, 1, 8, 200), (900, 2, 256, 384)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("perm", [False, True])
def test_forward_and_gradients(dev, dtype, size, perm):
    M, G, k, n = size
    say("grouped mm", size, dtype, "perm" if perm else "sorted")
    x, w, gy, off, p = make(M, G, k, n, dtype, perm, seed=M + 7 * k)
    groups = groups_of(off, p, dev)
    ref, s = blockref.grouped(x, w, off, p)
    xd, wd, gd = x.to(dev), w.to(dev), gy.to(dev)
    y = zs.zs_grouped_mm(xd, wd, groups)
    close(y, ref, blockref.sum_bound(ref, s, k, dtype), "y")
    gx, gw = zs.zs_grouped_mm_backward(gd, xd, wd, groups)
    ref, s = blockref.grouped(gy, w.transpose(1, 2), off, p)
    close(gx, ref, blockref.sum_bound(ref, s, n, dtype), "grad_x")
    ref, s = blockref.grouped_wgrad(x, gy, off, p, G)
    close(gw, ref, blockref.sum_bound(ref, s, M, dtype), "grad_w")
    # weights kept output-major: the same values through the transposed view, gradients of the same strides
    wt = wd.transpose(1, 2).contiguous().transpose(1, 2)
    ref, s = blockref.grouped(x, w, off, p)
    close(zs.zs_grouped_mm(xd, wt, groups), ref, blockref.sum_bound(ref, s, k, dtype), "y, w transposed")
    gx2, gw2 = zs.zs_grouped_mm_backward(gd, xd, wt, groups)
    ref, s = blockref.grouped(gy, w.transpose(1, 2), off, p)
    close(gx2, ref, blockref.sum_bound(ref, s, n, dtype), "grad_x, w transposed")
    ref, s = blockref.grouped_wgrad(x, gy, off, p, G)
    close(gw2, ref, blockref.sum_bound(ref, s, M, dtype), "grad_w, w transposed")
    # again: the same bits
    assert torch.equal(y, zs.zs_grouped_mm(xd, wd, groups))
    assert torch.equal(gw, zs.zs_grouped_mm_backward(gd, xd, wd, groups)[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(5000, 3, 32, 96), (20000, 2, 24, 40), (9000, 40, 64, 64)])
def test_long_groups_are_cut_and_joined(dev, dtype, shape):
    """Groups long enough that their rows are split over workgroups."""
    M, G, k, n = shape
    say("long groups", shape, dtype)
    x, w, gy, off, p = make(M, G, k, n, dtype, True, seed=M)
    gx, gw = zs.zs_grouped_mm_backward(gy.to(dev), x.to(dev), w.to(dev), groups_of(off, p, dev))
    ref, s = blockref.grouped_wgrad(x, gy, off, p, G)
    close(gw, ref, blockref.sum_bound(ref, s, M, dtype), "grad_w")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(3000, 511, 24, 40), (3000, 513, 24, 40), (5000, 2000, 72, 40), (300, 5000, 8, 136), (6000, 70000, 8, 8)])
def test_many_groups(dev, dtype, shape):
    """Around and above the number of groups whose tiles are counted, where a search finds a workgroup's group; more
    groups than rows; more than a grid's second dimension holds."""
    M, G, k, n = shape
    say("many groups", shape, dtype)
    rng = np.random.default_rng(G)
    x, w, gy, _, p = make(M, 1, k, n, dtype, True, seed=G)
    # few long groups among many short and empty ones
    at = np.sort(np.concatenate([rng.integers(0, M + 1, G - 1), [0, M]]))
    at[G // 2: G // 2 + G // 8] = at[G // 2]
    off = torch.from_numpy(at.astype(np.int32))
    w = torch.randn(1, k, n, generator=torch.Generator().manual_seed(1)).to(dtype).expand(G, k, n)
    groups = groups_of(off, p, dev)
    y = zs.zs_grouped_mm(x.to(dev), w.to(dev), groups)
    one = torch.tensor([0, M], dtype=torch.int32)   # equal weights: as one group
    ref, s = blockref.grouped(x, w[:1], one, p)
    close(y, ref, blockref.sum_bound(ref, s, k, dtype), "y")
    gx, gw = zs.zs_grouped_mm_backward(gy.to(dev), x.to(dev), w.to(dev), groups)
    ref, s = blockref.grouped(gy, w[:1].transpose(1, 2), one, p)
    close(gx, ref, blockref.sum_bound(ref, s, n, dtype), "grad_x")
    live = [g for g in range(G) if at[g + 1] > at[g]]
    assert (gw[torch.tensor([g for g in range(G) if at[g + 1] == at[g]], device=dev)] == 0).all()
    for g in live[:: max(1, len(live) // 200)] + [int(np.argmax(np.diff(at)))]:
        r = blockref.group_rows(off, p, g)
        ref, s = x[r].double().T @ gy[r].double(), x[r].double().abs().T @ gy[r].double().abs()
        close(gw[g], ref, blockref.sum_bound(ref, s, M, dtype), f"grad_w[{g}]")


def test_tile_shapes_of_large_products(dev):
    """bf16 products large enough for the tallest tiles, in one group (256 rows) and in uneven ones (192): rows against
    float64 at the ends of tiles and groups."""
    for M, G, k, n in ((16600, 1, 256, 4096), (16384, 7, 264, 2048), (9000, 3, 128, 8200)):
        say("large tiles", M, G, k, n)
        x, w, gy, off, p = make(M, G, k, n, BF16, True, seed=k, empty=False)
        y = zs.zs_grouped_mm(x.to(dev), w.to(dev), groups_of(off, p, dev)).cpu()
        pos = torch.unique(torch.cat([off.long()[:-1], off.long()[1:] - 1, torch.arange(0, M, 191), torch.arange(M - 300, M)]))
        group = torch.searchsorted(off[1:].long(), pos, right=True)
        rows = p[pos].long()
        for g in range(G):
            r = rows[group == g]
            ref, s = x[r].double() @ w[g].double(), x[r].double().abs() @ w[g].double().abs()
            close(y[r], ref, blockref.sum_bound(ref, s, k, BF16), f"group {g}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_past_32_bits(dev, dtype):
    """Rows whose elements lie more than 2^32 elements from the start, in x, grad_y and the output, and weights of
    groups that far apart."""
    M, G, k, n = 700, 2, 40, 24
    stride = 1 << 23
    say("wide offsets", dtype)
    x, w, gy, off, p = make(M, G, k, n, dtype, True, seed=21, empty=False)
    groups = groups_of(off, p, dev)
    size = (M - 1) * stride + 64
    assert size > 1 << 32
    big = torch.empty(size, dtype=dtype, device=dev)
    xv, gv, yv = (big.as_strided((M, c), (stride, 1), at) for c, at in ((k, 0), (n, 0), (n, 0)))
    ref, s = blockref.grouped(x, w, off, p)
    xv.copy_(x.to(dev))
    close(zs.zs_grouped_mm(xv, w.to(dev), groups), ref, blockref.sum_bound(ref, s, k, dtype), "y")
    gref, gs = blockref.grouped_wgrad(x, gy, off, p, G)
    close(zs.zs_grouped_mm_backward(gy.to(dev), xv, w.to(dev), groups)[1], gref, blockref.sum_bound(gref, gs, M, dtype), "grad_w")
    zs.zs_grouped_mm(x.to(dev), w.to(dev), groups, out=yv)
    close(yv, ref, blockref.sum_bound(ref, s, k, dtype), "y, wide")
    gv.copy_(gy.to(dev))
    gx, gw = zs.zs_grouped_mm_backward(gv, x.to(dev), w.to(dev), groups)
    close(gw, gref, blockref.sum_bound(gref, gs, M, dtype), "grad_w, wide grad_y")
    xref, xs = blockref.grouped(gy, w.transpose(1, 2), off, p)
    close(gx, xref, blockref.sum_bound(xref, xs, n, dtype), "grad_x, wide grad_y")
    far = big.as_strided((G, k, n), (size - k * n, n, 1))
    far.copy_(w.to(dev))
    close(zs.zs_grouped_mm(x.to(dev), far, groups), ref, blockref.sum_bound(ref, s, k, dtype), "y, far weights")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("perm", [False, True])
def test_rows_of_no_group_get_zeros(dev, dtype, perm):
    M, G, k, n = 400, 5, 48, 72
    say("rows outside", dtype, perm)
    x, w, gy, off, p = make(M, G, k, n, dtype, perm, seed=3, outside=True)
    groups = groups_of(off, p, dev)
    x[:3] = float("nan") if not perm else x[:3]   # before the first offset: not read into any result
    y = zs.zs_grouped_mm(x.to(dev), w.to(dev), groups)
    rows = torch.cat([torch.arange(0, int(off[0])), torch.arange(int(off[-1]), M)])
    rows = rows if p is None else p[rows].long()
    assert rows.numel() > 100 and (y[rows.to(dev)] == 0).all()
    x = torch.nan_to_num(x)
    ref, s = blockref.grouped(x, w, off, p)
    close(zs.zs_grouped_mm(x.to(dev), w.to(dev), groups), ref, blockref.sum_bound(ref, s, k, dtype), "y")
    # a set of only empty groups
    none = groups_of(torch.zeros(G + 1, dtype=torch.int32), p, dev)
    assert (zs.zs_grouped_mm(x.to(dev), w.to(dev), none) == 0).all()
    gx, gw = zs.zs_grouped_mm_backward(gy.to(dev), x.to(dev), w.to(dev), none)
    assert (gx == 0).all() and (gw == 0).all()


def test_no_rows(dev):
    say("no rows")
    groups = groups_of(torch.zeros(4, dtype=torch.int32), None, dev)
    x, w = torch.empty(0, 8, device=dev), torch.ones(3, 8, 5, device=dev)
    assert zs.zs_grouped_mm(x, w, groups).shape == (0, 5)
    gx, gw = zs.zs_grouped_mm_backward(torch.empty(0, 5, device=dev), x, w, groups)
    assert gx.shape == (0, 8) and gw.shape == (3, 8, 5) and (gw == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(130, 3, 16, 33, 40), (130, 3, 16, 36, 44), (700, 3, 40, 93, 96), (9000, 4, 64, 1021, 1024),
                                  (9000, 2, 64, 2041, 2056), (33, 2, 24, 7, 8)])
@pytest.mark.parametrize("perm", [False, True])
def test_odd_widths_into_padded_rows(dev, dtype, size, perm):
    """Columns that end inside 16 bytes of a row that starts on 16 bytes: the padding behind them, rows of no group
    and the rows around the output."""
    M, G, k, n, stride = size
    say("padded rows", dtype, size, perm)
    x, w, gy, off, p = make(M, G, k, n, dtype, perm, seed=n, outside=True)
    ob = torch.full((M + 2, stride), 77.0, dtype=dtype, device=dev)
    y = zs.zs_grouped_mm(x.to(dev), w.transpose(1, 2).contiguous().to(dev).transpose(1, 2), groups_of(off, p, dev),
                         out=ob[1:-1, :n])
    ref, s = blockref.grouped(x, w, off, p)
    close(y, ref, blockref.sum_bound(ref, s, k, dtype), "y")
    assert (ob[0] == 77).all() and (ob[-1] == 77).all() and (ob[:, n:] == 77).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [1, 8])
def test_strided_views_and_guards(dev, dtype, pad):
    """Row-strided x and grad_y (aligned and unaligned strides and starts) read in place, a strided output whose
    padding keeps its values, broadcast rows."""
    M, G, k, n = 260, 3, 64, 96
    say("strided", dtype, pad)
    x, w, gy, off, p = make(M, G, k, n, dtype, True, seed=11)
    groups = groups_of(off, p, dev)
    xb = torch.full((M, k + 2 * pad), float("nan"), dtype=dtype, device=dev)
    xb[:, pad:pad + k] = x.to(dev)
    gb = torch.full((M, n + 2 * pad), float("nan"), dtype=dtype, device=dev)
    gb[:, pad:pad + n] = gy.to(dev)
    ob = torch.full((M + 2, n + pad), 77.0, dtype=dtype, device=dev)
    y = zs.zs_grouped_mm(xb[:, pad:pad + k], w.to(dev), groups, out=ob[1:-1, :n])
    ref, s = blockref.grouped(x, w, off, p)
    close(y, ref, blockref.sum_bound(ref, s, k, dtype), "y")
    assert (ob[0] == 77).all() and (ob[-1] == 77).all() and (ob[:, n:] == 77).all()
    gx, gw = zs.zs_grouped_mm_backward(gb[:, pad:pad + n], xb[:, pad:pad + k], w.to(dev), groups)
    ref, s = blockref.grouped(gy, w.transpose(1, 2), off, p)
    close(gx, ref, blockref.sum_bound(ref, s, n, dtype), "grad_x")
    ref, s = blockref.grouped_wgrad(x, gy, off, p, G)
    close(gw, ref, blockref.sum_bound(ref, s, M, dtype), "grad_w")
    one = x[:1].expand(M, k)
    ref, s = blockref.grouped(one, w, off, p)
    close(zs.zs_grouped_mm(x[:1].to(dev).expand(M, k), w.to(dev), groups), ref, blockref.sum_bound(ref, s, k, dtype), "y of one row")
    shared = w[:1].expand(G, k, n)   # one weight for all groups
    ref, s = blockref.grouped(x, shared, off, p)
    close(zs.zs_grouped_mm(x.to(dev), w[:1].to(dev).expand(G, k, n), groups), ref, blockref.sum_bound(ref, s, k, dtype), "y of one weight")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_non_finite_rows_stay_in_their_rows(dev, dtype):
    """An infinite or NaN row spoils its own output row and its group's weight gradient only, at widths with partial
    tiles."""
    M, G, k, n = 200, 3, 40, 56
    say("non-finite", dtype)
    x, w, gy, off, _ = make(M, G, k, n, dtype, False, seed=5, empty=False)
    w = w.abs() + 0.5
    x[10] = x[10].abs() + 1
    x[10, 3] = float("inf")
    x[20, 7] = float("nan")
    groups = groups_of(off, None, dev)
    y = zs.zs_grouped_mm(x.to(dev), w.to(dev), groups).cpu()
    assert torch.isinf(y[10]).all() and (y[10] > 0).all() and torch.isnan(y[20]).all()
    rest = [i for i in range(M) if i not in (10, 20)]
    assert torch.isfinite(y[rest]).all()
    gw = zs.zs_grouped_mm_backward(gy.to(dev), x.to(dev), w.to(dev), groups)[1].cpu()
    assert torch.isfinite(gw[1:]).all() and not torch.isfinite(gw[0, 3]).all()
    assert torch.isfinite(gw[0, [i for i in range(k) if i not in (3, 7)]]).all()


def test_built_csr_gives_the_groups(dev):
    """zs_build_csr over the rows' species is the grouping; autograd through grouped_mm, the gradient against
    differences of the float64 product."""
    M, G, k, n = 777, 6, 24, 40
    say("csr groups, autograd")
    gen = torch.Generator().manual_seed(1)
    species = torch.randint(0, G, (M,), generator=gen)
    species[species == 2] = 3
    csr = zs.zs_build_csr(species.to(dev), G)
    x, w = torch.randn(M, k, generator=gen), torch.randn(G, k, n, generator=gen)
    xd, wd = x.to(dev).requires_grad_(), w.to(dev).requires_grad_()
    y = zs.grouped_mm(xd, wd, csr)
    ref = torch.bmm(x.double()[:, None], w.double()[species])[:, 0]
    assert (y.double().cpu() - ref).abs().max() <= 40 * 2.0 ** -23 * k
    c = torch.randn(M, n, generator=gen)
    (y * c.to(dev)).sum().backward()
    assert (wd.grad[2] == 0).all()
    dx, dw = torch.randn(M, k, generator=gen).double(), torch.randn(G, k, n, generator=gen).double()
    f = lambda t: (torch.bmm((x.double() + t * dx)[:, None], (w.double() + t * dw)[species])[:, 0] * c.double()).sum()  # noqa: E731
    slope = (f(1e-4) - f(-1e-4)) / 2e-4
    got = (xd.grad.double().cpu() * dx).sum() + (wd.grad.double().cpu() * dw).sum()
    # the product is bilinear, so the central difference is exact up to float64 rounding; each gradient entry is a
    # sum of at most 777 terms
    scale = (xd.grad.abs().double().cpu() * dx.abs()).sum() + (wd.grad.abs().double().cpu() * dw.abs()).sum()
    assert abs(got - slope) <= 800 * 2.0 ** -23 * scale
    lin = zs.grouped_mm(xd, wd, csr).sum()
    assert torch.autograd.grad(lin, xd, retain_graph=False)[0].shape == xd.shape


def test_side_stream_and_graph(dev):
    """Calls on a stream of their own, and captured in a graph whose replays follow changed inputs."""
    M, G, k, n = 3000, 4, 32, 96
    say("stream and graph")
    x, w, gy, off, p = make(M, G, k, n, F32, True, seed=9)
    xd, wd, gd, groups = x.to(dev), w.to(dev), gy.to(dev), groups_of(off, p, dev)
    want = zs.zs_grouped_mm(xd, wd, groups), *zs.zs_grouped_mm_backward(gd, xd, wd, groups)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = zs.zs_grouped_mm(xd, wd, groups), *zs.zs_grouped_mm_backward(gd, xd, wd, groups)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = zs.zs_grouped_mm(xd, wd, groups), *zs.zs_grouped_mm_backward(gd, xd, wd, groups)
    for i in range(4):
        xd.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        want = zs.zs_grouped_mm(xd, wd, groups), *zs.zs_grouped_mm_backward(gd, xd, wd, groups)
        assert all(torch.equal(a, b) for a, b in zip(want, res)), i


def test_refusals(dev):
    say("refusals")
    x, w = torch.zeros(10, 8, device=dev), torch.zeros(2, 8, 4, device=dev)
    g = groups_of(torch.tensor([0, 4, 10], dtype=torch.int32), None, dev)
    with pytest.raises(ValueError):
        zs.zs_grouped_mm(x.cpu(), w, g)
    with pytest.raises(TypeError):
        zs.zs_grouped_mm(x.half(), w.half(), g)
    with pytest.raises(TypeError):
        zs.zs_grouped_mm(x, w.bfloat16(), g)
    with pytest.raises(ValueError):
        zs.zs_grouped_mm(x[:, :7], w, g)
    with pytest.raises(ValueError):
        zs.zs_grouped_mm(x, w[:1], g)
    with pytest.raises(ValueError):
        zs.zs_grouped_mm(x, w, g, out=torch.empty(10, 5, device=dev))
    with pytest.raises(ValueError):
        zs.zs_grouped_mm(x, w, g._replace(perm=torch.zeros(9, dtype=torch.int32, device=dev)))
    with pytest.raises(TypeError):
        zs.zs_grouped_mm(x, w, g._replace(rowptr=g.rowptr.long()))
    with pytest.raises(zs.ZsError):   # output over the input
        zs.zs_grouped_mm(x, torch.zeros(2, 8, 8, device=dev), g, out=x)
    with pytest.raises(ValueError):
        zs.zs_grouped_mm_backward(torch.zeros(10, 5, device=dev), x, w, g)


def test_output_counts_as_written(dev):
    """Writing `out` counts as a change of it: a graph that saved its values refuses its backward."""
    x, w = torch.ones(4, 8, device=dev), torch.ones(1, 8, 8, device=dev, requires_grad=True)
    groups = groups_of(torch.tensor([0, 4], dtype=torch.int32), None, dev)
    out = torch.ones(4, 8, device=dev)
    before = out._version
    loss = (out * zs.grouped_mm(x, w, groups)).sum()
    zs.zs_grouped_mm(x, w.detach(), groups, out=out)
    assert out._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_workgroups_than_one_launch_holds(dev, dtype):
    """A launch has less than 2^32 threads.  The most groups, few of them with rows, and columns enough for 2^24
    workgroups: windows of one array as the groups' weights (each group its own), and a weight gradient of 2 or 4 GiB."""
    M, G, k, n = 1000, 1 << 20, 8, 2048
    say("many workgroups", dtype)
    rng = np.random.default_rng(7)
    gen = torch.Generator().manual_seed(7)
    at = np.sort(np.concatenate([rng.integers(0, M + 1, G - 1), [0, M]]))
    at[:G // 3] = 0   # the first rows belong to a group far behind
    off = torch.from_numpy(at.astype(np.int32))
    p = torch.from_numpy(rng.permutation(M).astype(np.int32))
    groups = groups_of(off, p, dev)
    x = torch.randint(-2, 3, (M, k), generator=gen).to(dtype)
    base = torch.randint(-2, 3, (G * 8 + k * n,), generator=gen).to(dtype).to(dev)
    y = zs.zs_grouped_mm(x.to(dev), base.as_strided((G, k, n), (8, n, 1)), groups).cpu()
    pos = torch.searchsorted(off[1:].long(), torch.arange(M), right=True)
    base = base.cpu()
    for i in range(M):
        r, g = int(p[i]), int(pos[i])
        want = x[r].double() @ base.as_strided((k, n), (n, 1), g * 8).double()
        assert torch.equal(y[r], want.to(dtype)), (i, g)
    del base, y
    k, n = 1, 1024
    x, gy = (torch.randint(-2, 3, s, generator=gen).to(dtype) for s in ((M, k), (M, n)))
    stale = torch.full((G, k, n), 7.0, dtype=dtype, device=dev)   # the memory the gradient then gets
    w = torch.ones(1, k, n, dtype=dtype, device=dev).expand(G, k, n)
    del stale
    gx, gw = zs.zs_grouped_mm_backward(gy.to(dev), x.to(dev), w, groups)
    assert torch.equal(gx.cpu(), gy.double().sum(1, keepdim=True).to(dtype))
    live = torch.unique(pos)
    want = torch.zeros(len(live), k, n, dtype=torch.float64)
    for j, g in enumerate(live.tolist()):
        r = blockref.group_rows(off, p, g)
        want[j] = x[r].double().T @ gy[r].double()
    assert torch.equal(gw[live.to(dev)].cpu(), want.to(dtype))
    gw[live.to(dev)] = 0
    assert gw.count_nonzero().item() == 0


def test_output_of_one_row(dev):
    """The stride of a single row's dimension says nothing: a column's transpose is such an output."""
    x, w = torch.ones(1, 8, device=dev), torch.ones(2, 8, 24, device=dev)
    groups = groups_of(torch.tensor([0, 1, 1], dtype=torch.int32), None, dev)
    out = torch.zeros(24, 1, device=dev).t()
    assert out.stride(0) < 24
    zs.zs_grouped_mm(x, w, groups, out=out)
    assert (out == 8).all()


def whole(M, G, k, n, dtype, perm, seed, empty=True):
    """make() with whole numbers of at most 2: every sum below 2^24 is exact in fp32, so results are the definition's
    rounded once and have to be equal to it."""
    _, _, _, off, p = make(M, G, 1, 1, dtype, perm, seed, empty)
    gen = torch.Generator().manual_seed(seed)
    assert 4 * max(M, k, n) < 1 << 24
    mk = lambda *s: torch.randint(-2, 3, s, generator=gen).to(dtype)  # noqa: E731
    return mk(M, k), mk(G, k, n), mk(M, n), off, p


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(5000, 3, 32, 96), (20000, 2, 24, 40), (9000, 40, 64, 64), (9000, 3, 776, 1160), (9000, 3, 777, 1161), (900000, 2, 32, 96)])
@pytest.mark.parametrize("perm", [False, True])
def test_cut_groups_exactly(dev, dtype, shape, perm):
    """Both gradients where groups are cut into pieces: pieces longer than the 1024 row indices that a workgroup holds
    at a time (the last three; 1230 rows and 1172), wide weights whose tiles are spread over the XCDs, operands off 16
    bytes, and the one pass of narrow weights."""
    M, G, k, n = shape
    say("cut groups", shape, dtype, "perm" if perm else "sorted")
    x, w, gy, off, p = whole(M, G, k, n, dtype, perm, seed=k)
    groups = groups_of(off, p, dev)
    gx, gw = zs.zs_grouped_mm_backward(gy.to(dev), x.to(dev), w.to(dev), groups)
    alone = zs.zs_grouped_mm_backward(gy.to(dev), x.to(dev), w.to(dev), groups, need_x=False)[1]
    for g in range(G):
        r = blockref.group_rows(off, p, g)
        a, b = x[r].double(), gy[r].double()
        want = (a.T @ b).to(dtype)
        assert torch.equal(gw[g].cpu(), want), f"grad_w of group {g}"
        assert torch.equal(alone[g].cpu(), want), f"grad_w of group {g}, alone"
        assert torch.equal(gx[r.to(dev)].cpu(), (b @ w[g].double().T).to(dtype)), f"grad_x of group {g}"
