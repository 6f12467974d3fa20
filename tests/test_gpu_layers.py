"""Lookup by token or species, layer norm and the weighted sum of experts' rows, with their gradients, against float64
on the GPU."""
import pytest
import torch

import edge_node_scatter_amd as zs
import layersref as ref
from edge_node_scatter_amd import layers

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
WIDTHS = [1, 3, 8, 30, 64, 129, 257, 520, 777, 1024, 1032, 1540, 2048, 4100, 8192]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.load()
    return torch.device("cuda:0")


def say(*a):
    print("[gpu]", *a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def mk(g, *s, std=1.0, dtype=F32):
    return (std * torch.randn(*s, generator=g)).to(dtype)


def within(got, want, bound, what):
    got, over = got.double().cpu(), None
    assert got.shape == want.shape, what
    over = (got - want).abs() - bound
    assert not got.isnan().any() and (over <= 0).all(), f"{what}: {over.max().item()} over the bound"


def bits(*ts):
    return [t.view(torch.int32 if t.dtype == F32 else torch.int16 if t.dtype == BF16 else t.dtype) for t in ts]


# ---- lookup -----------------------------------------------------------------------------------------------------

def tokens(g, M, V, pad=True):
    """Indices whose frequencies fall with the rank, some outside the table."""
    p = 1 / torch.arange(1, V + 1, dtype=torch.float64)
    index = torch.randperm(V, generator=g)[torch.multinomial(p, max(M, 1), replacement=True, generator=g)[:M]]
    if pad and M:
        index[torch.rand(M, generator=g) < 0.1] = -1
        index[0] = V
        index[-1] = -(1 << 40)
    return index


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", WIDTHS)
def test_embedding(dev, dtype, c):
    for M, V in ((0, 5), (1, 1), (7, 300), (533, 40)):
        say("embedding", dtype, M, V, c)
        g = gen(M + c)
        table, index = mk(g, V, c, dtype=dtype), tokens(g, M, V, pad=M > 2)
        for scale in (1.0, -0.37):
            want, bound = ref.embedding(table, index, scale)
            within(zs.zs_embedding(table.to(dev), index.to(dev), scale), want, bound(dtype), (M, V, scale))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embedding_of_many_rows(dev, dtype):
    """Row counts on both sides of every choice of rows a turn."""
    for M, c in ((4095 * 8, 256), (4096 * 8 + 3, 256), (70001, 8), (20000, 2048)):
        say("embedding rows", dtype, M, c)
        g = gen(M)
        table, index = mk(g, 97, c, dtype=dtype), tokens(g, M, 97)
        want, bound = ref.embedding(table, index, 0.5)
        within(zs.zs_embedding(table.to(dev), index.to(dev), 0.5), want, bound(dtype), (M, c))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embedding_layouts(dev, dtype):
    say("embedding layouts", dtype)
    g = gen(3)
    big, index = mk(g, 50, 200, dtype=dtype).to(dev), tokens(g, 91, 40).to(dev)
    for t in (big[:40, :64], big[:40, 3:67], big[5:45, 1:], big.T[:40, :33], big[:1, :64].expand(40, 64), big[:40, :1].expand(40, 24)):
        want, bound = ref.embedding(t.cpu(), index.cpu(), 2.0)
        within(zs.zs_embedding(t, index, 2.0), want, bound(dtype), t.stride())
    double = torch.stack([index, index], 1)[:, 0]   # a strided index
    assert torch.equal(zs.zs_embedding(big[:40], double), zs.zs_embedding(big[:40], index))
    # padding is +0 whatever the scale, and what is not a number comes back as it is
    t = torch.full((3, 16), float("nan"), dtype=dtype, device=dev)
    t[1] = float("inf")
    y = zs.zs_embedding(t, torch.tensor([-1, 1, 0, 3], device=dev), -2.0)
    assert (y[0] == 0).all() and not y[0].signbit().any() and (y[1] == -float("inf")).all() and y[2].isnan().all() and (y[3] == 0).all()


def sorted_form(index, V):
    """(rows in order, offsets) of indices inside [0, V)."""
    order = torch.argsort(index, stable=True)
    return order, torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(index, minlength=V).cumsum(0)]).to(torch.int32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", WIDTHS)
def test_embedding_backward(dev, dtype, c):
    for M, V in ((0, 5), (1, 1), (9, 300), (1500, 3), (2100, 70), (2100, 1024), (900, 1500)):
        say("embedding backward", dtype, M, V, c)
        g = gen(M + 7 * c)
        gy, index = mk(g, M, c, dtype=dtype), tokens(g, M, V, pad=M > 2)
        want, bound = ref.embedding_grad(gy, index, V, 0.7)
        got = zs.zs_embedding_backward(gy.to(dev), index.to(dev), V, 0.7)
        within(got, want, bound(dtype), (M, V))
        assert all(torch.equal(a, b) for a, b in zip(bits(got), bits(zs.zs_embedding_backward(gy.to(dev), index.to(dev), V, 0.7))))
        if M > 2:
            inside = index.clamp(0, V - 1)
            groups = zs.zs_build_csr(inside.to(dev), V)
            want, bound = ref.embedding_grad(gy, inside, V, 0.7)
            within(zs.zs_embedding_backward(gy.to(dev), inside.to(dev), V, 0.7, groups), want, bound(dtype), "groups")


@pytest.mark.parametrize("dtype,c", [(F32, 32), (BF16, 32), (F32, 4), (BF16, 8), (BF16, 1), (BF16, 512), (F32, 300), (BF16, 1100)])
def test_embedding_backward_of_runs(dev, dtype, c):
    """Runs that end where a lane's, a workgroup's or several workgroups' positions do, runs of one row, one run of all."""
    for sizes in ([8, 8, 16, 1, 7, 32, 64, 64, 128, 256, 512, 1024, 2048, 4096, 2048, 1, 1, 1, 5], [20011], [0, 0, 20480, 0], [1] * 3000, [2047, 2, 2047, 4097, 0, 8191],
                  [1, 0, 0, 1] + [0] * 4000 + [9000], [64] * 200, [3, 61] * 100, [255, 257, 1, 511]):
        say("runs", dtype, c, len(sizes), sum(sizes))
        V, M = len(sizes), sum(sizes)
        index = torch.repeat_interleave(torch.arange(V), torch.tensor(sizes))
        gy = mk(gen(M), M, c, dtype=dtype)
        offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.tensor(sizes).cumsum(0)]).to(torch.int32)
        want, bound = ref.embedding_grad(gy, index, V, 1.0)
        got = zs.zs_embedding_backward(gy.to(dev), index.to(dev), V, 1.0, zs.sorted_groups(offsets.to(dev)))
        within(got, want, bound(dtype), sizes[:4])
        assert (got.cpu()[torch.tensor(sizes) == 0] == 0).all()
        perm = torch.randperm(M, generator=gen(1))
        got = zs.zs_embedding_backward(gy[perm].to(dev), index[perm].to(dev), V)
        within(got, want, bound(dtype), "in any order")


def test_embedding_backward_of_all_padding(dev):
    say("all padding")
    for M in (1, 5000):
        got = zs.zs_embedding_backward(torch.ones(M, 24, device=dev), torch.full((M,), -1, device=dev), 33)
        assert got.shape == (33, 24) and (got == 0).all()


def test_embedding_backward_layouts(dev):
    say("embedding backward layouts")
    g = gen(5)
    big, index = mk(g, 700, 200).to(dev), tokens(g, 600, 20).to(dev)
    for gy in (big[:600, :64], big[:600, 3:70], big.T[:, :600].T[:, :50], big[:1, :64].expand(600, 64), big[:600, :1].expand(600, 40)):
        want, bound = ref.embedding_grad(gy.cpu(), index.cpu(), 20, 1.5)
        within(zs.zs_embedding_backward(gy, index, 20, 1.5), want, bound(F32), gy.stride())


def test_embedding_offsets_that_do_not_fit_the_index(dev):
    """Groups of another index: values are unspecified, memory behind the arrays is not touched."""
    say("foreign groups")
    lib, M, V, c = layers.load_layers(), 3000, 50, 40
    index = torch.randint(-3, V + 3, (M,), generator=gen(2)).to(dev)
    gy = torch.ones(M, c, device=dev)
    size = lib.zs_embedding_backward_workspace_bytes(M, c, 0)
    for offsets, perm in ((torch.randint(-100, 2 * M, (V + 1,), generator=gen(3)), torch.randint(-5, M + 5, (M,), generator=gen(4))),
                          (torch.arange(V, -1, -1) * 60, torch.zeros(M)), (torch.full((V + 1,), 1 << 30), torch.arange(M))):
        out, ws = torch.full((V + 2, c), 7.0, device=dev), torch.full((size + 256,), 9, dtype=torch.uint8, device=dev)
        o, p = offsets.to(torch.int32).to(dev), perm.to(torch.int32).to(dev)
        st = zs._call(dev, lib.zs_embedding_backward, gy.data_ptr(), c, index.data_ptr(), o.data_ptr(), p.data_ptr(), M, V, c, 1.0, 0, out[1:].data_ptr(), ws.data_ptr(), size)
        torch.cuda.synchronize()
        assert st == 0 and (out[0] == 7).all() and (out[-1] == 7).all() and (ws[size:] == 9).all()


def test_csr_leaves_padding_out(dev):
    """Entries outside the nodes: counted nowhere, and the others stand first in perm."""
    say("csr with padding")
    for M, V in ((5000, 37), (3, 2), (4100, 70000), (9000, 600000)):
        index = tokens(gen(M), M, V)
        flag = torch.zeros(1, dtype=torch.int32, device=dev)
        csr = zs.zs_build_csr(index.to(dev), V, bad_flag=flag, order=False)
        live = (index >= 0) & (index < V)
        order = torch.arange(M)[live][torch.argsort(index[live], stable=True)]
        assert flag.item() != 0
        assert torch.equal(csr.rowptr.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(index[live], minlength=V).cumsum(0)]))
        assert torch.equal(csr.perm.cpu().long()[:order.numel()], order)


# ---- layer norm -------------------------------------------------------------------------------------------------

def norm_inputs(M, c, dtype, seed, shift=0.0):
    g = gen(seed)
    return mk(g, M, c, std=1.5).add_(shift).to(dtype), 1 + 0.2 * mk(g, c), 0.3 * mk(g, c), mk(g, M, c, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", WIDTHS)
def test_layer_norm(dev, dtype, c):
    for M in (0, 1, 5, 300):
        say("layer norm", dtype, M, c)
        x, w, b, gy = norm_inputs(M, c, dtype, M + c)
        for bias in (b, None):
            want, bound = ref.layer_norm(x, w, bias, 1e-5)
            within(zs.zs_layer_norm(x.to(dev), w.to(dev), None if bias is None else bias.to(dev)), want, bound(dtype), (M, bias is None))
        (gx, gw, gb), (bx, bw, bb) = ref.layer_norm_grads(gy, x, w, 1e-5)
        for need in (True, False):
            got = zs.zs_layer_norm_backward(gy.to(dev), x.to(dev), w.to(dev), need)
            within(got[0], gx, bx(dtype), "grad_x")
            within(got[1], gw, bw() if M else torch.zeros(c), "grad_w")
            assert (got[2] is None) == (not need)
            if need:
                within(got[2], gb, bb() if M else torch.zeros(c), "grad_b")
        again = zs.zs_layer_norm_backward(gy.to(dev), x.to(dev), w.to(dev))
        first = zs.zs_layer_norm_backward(gy.to(dev), x.to(dev), w.to(dev))
        assert all(torch.equal(a, b) for a, b in zip(bits(*first), bits(*again)))


@pytest.mark.parametrize("dtype,M,c", [(F32, 40000, 32), (BF16, 9001, 520), (F32, 3001, 777), (BF16, 2100, 2048), (F32, 1300, 8192)])
def test_layer_norm_of_many_rows(dev, dtype, M, c):
    """More rows than one round of workgroups."""
    say("layer norm rows", dtype, M, c)
    x, w, b, gy = norm_inputs(M, c, dtype, M)
    want, bound = ref.layer_norm(x, w, b, 1e-5)
    within(zs.zs_layer_norm(x.to(dev), w.to(dev), b.to(dev)), want, bound(dtype), "y")
    (gx, gw, gb), (bx, bw, bb) = ref.layer_norm_grads(gy, x, w, 1e-5)
    got = zs.zs_layer_norm_backward(gy.to(dev), x.to(dev), w.to(dev))
    within(got[0], gx, bx(dtype), "grad_x")
    within(got[1], gw, bw(), "grad_w")
    within(got[2], gb, bb(), "grad_b")


def test_layer_norm_of_odd_rows(dev):
    say("layer norm, odd rows")
    w, b = torch.ones(257), torch.zeros(257)
    # a mean far above the spread: fp32 inputs hold the spread exactly
    x = (4096 + torch.randint(-8, 9, (40, 257), generator=gen(1)) * 0.125).float()
    want, bound = ref.layer_norm(x, w, b, 1e-5)
    within(zs.zs_layer_norm(x.to(dev), w.to(dev), b.to(dev)), want, bound(F32), "far mean")
    gy = mk(gen(2), 40, 257)
    (gx, _, _), (bx, _, _) = ref.layer_norm_grads(gy, x, w, 1e-5)
    within(zs.zs_layer_norm_backward(gy.to(dev), x.to(dev), w.to(dev))[0], gx, bx(F32), "far mean")
    # constant rows, tiny and large values, one channel
    for x in (torch.full((3, 257), 3.0), 1e-12 * mk(gen(3), 5, 257), 1e15 * mk(gen(4), 5, 257)):
        want, bound = ref.layer_norm(x, w, b, 1e-5)
        within(zs.zs_layer_norm(x.to(dev), w.to(dev), b.to(dev)), want, bound(F32), "scale")
        (gx, _, _), (bx, _, _) = ref.layer_norm_grads(gy[:x.shape[0]], x, w, 1e-5)
        within(zs.zs_layer_norm_backward(gy[:x.shape[0]].to(dev), x.to(dev), w.to(dev))[0], gx, bx(F32), "scale")
    # constant rows whose sum is not exact: no spread, so nothing that is not a number
    for v in (1.1e6, 7.3e9, 3.3e15):
        for c in (30, 257, 777, 1031, 2048, 4100):
            x, one = torch.full((5, c), v, device=dev), torch.ones(c, device=dev)
            assert zs.zs_layer_norm(x, one).isfinite().all()
            assert all(t.isfinite().all() for t in zs.zs_layer_norm_backward(torch.ones_like(x), x, one))
    y = zs.zs_layer_norm(torch.tensor([[5.0], [-2.0]], device=dev), torch.ones(1, device=dev), torch.full((1,), 0.25, device=dev))
    assert (y == 0.25).all()
    # what is not a number stays in its row
    x = mk(gen(5), 9, 257)
    x[2, 7], x[5, 3] = float("nan"), float("inf")
    y = zs.zs_layer_norm(x.to(dev), w.to(dev), b.to(dev)).cpu()
    gx = zs.zs_layer_norm_backward(gy[:9].to(dev), x.to(dev), w.to(dev))[0].cpu()
    rows = torch.tensor([0, 1, 3, 4, 6, 7, 8])
    assert y[2].isnan().all() and y[5].isnan().all() and gx[2].isnan().all()
    want, bound = ref.layer_norm(x[rows], w, b, 1e-5)
    within(y[rows], want, bound(F32), "the other rows")


def test_layer_norm_layouts(dev):
    say("layer norm layouts")
    g = gen(8)
    big, w, b = mk(g, 300, 300).to(dev), 1 + 0.2 * mk(g, 300), mk(g, 300)
    gy = mk(g, 300, 300).to(dev)
    for sl in ((slice(0, 90), slice(0, 64)), (slice(3, 99), slice(5, 134)), (slice(0, 90), slice(0, 1))):
        for x, t in ((big[sl], gy[sl]), (big.T[sl], gy[sl]), (big[sl], gy.T[sl]), (big[:1].expand(300, 300)[sl], gy[sl]), (big[sl], gy[:1, :1].expand(300, 300)[sl])):
            c = x.shape[1]
            want, bound = ref.layer_norm(x.cpu(), w[:c], b[:c], 1e-3)
            within(zs.zs_layer_norm(x, w[:c].to(dev), b.to(dev)[1:c + 1] * 0 + b[:c].to(dev), eps=1e-3), want, bound(F32), x.stride())
            (gx, gw, gb), (bx, bw, bb) = ref.layer_norm_grads(t.cpu(), x.cpu(), w[:c], 1e-3)
            got = zs.zs_layer_norm_backward(t, x, w.to(dev)[:c], eps=1e-3)
            within(got[0], gx, bx(F32), "grad_x")
            within(got[1], gw, bw(), "grad_w")
            within(got[2], gb, bb(), "grad_b")
    # parameters that start anywhere
    wide = torch.stack([w, b]).to(dev)
    y = zs.zs_layer_norm(big[:50, :128], wide[0, 1:129], wide[1, 3:131])
    want, bound = ref.layer_norm(big[:50, :128].cpu(), w[1:129], b[3:131], 1e-5)
    within(y, want, bound(F32), "offset parameters")


# ---- weighted sum -----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", WIDTHS)
def test_combine(dev, dtype, c):
    for M, k in ((0, 2), (1, 1), (1, 64), (7, 3), (130, 8), (41, 6)):
        say("combine", dtype, M, k, c)
        g = gen(M + c + k)
        z, weight, gy = mk(g, M * k, c, dtype=dtype), mk(g, M, k), mk(g, M, c, dtype=dtype)
        want, bound = ref.combine(z, weight)
        within(zs.zs_combine(z.to(dev), weight.to(dev)), want, bound(dtype), (M, k))
        (gz, gw), (bz, bw) = ref.combine_grads(gy, z, weight)
        got = zs.zs_combine_backward(gy.to(dev), z.to(dev), weight.to(dev))
        within(got[0], gz, bz(dtype), "grad_z")
        within(got[1], gw, bw(), "grad_weight")
        again = zs.zs_combine_backward(gy.to(dev), z.to(dev), weight.to(dev))
        assert all(torch.equal(a, b) for a, b in zip(bits(*got), bits(*again)))


@pytest.mark.parametrize("dtype,M,k,c", [(F32, 9000, 2, 520), (BF16, 8200, 3, 2048), (BF16, 70000, 4, 8), (F32, 8300, 2, 4100)])
def test_combine_of_many_rows(dev, dtype, M, k, c):
    say("combine rows", dtype, M, k, c)
    g = gen(M)
    z, weight, gy = mk(g, M * k, c, dtype=dtype), mk(g, M, k), mk(g, M, c, dtype=dtype)
    want, bound = ref.combine(z, weight)
    within(zs.zs_combine(z.to(dev), weight.to(dev)), want, bound(dtype), "y")
    (gz, gw), (bz, bw) = ref.combine_grads(gy, z, weight)
    got = zs.zs_combine_backward(gy.to(dev), z.to(dev), weight.to(dev))
    within(got[0], gz, bz(dtype), "grad_z")
    within(got[1], gw, bw(), "grad_weight")


def test_combine_layouts(dev):
    say("combine layouts")
    g = gen(9)
    big, gyb, weight = mk(g, 300, 300).to(dev), mk(g, 300, 300).to(dev), mk(g, 30, 6).to(dev)
    for z, gy, w in ((big[:180, :64], gyb[:30, :64], weight), (big[9:189, 3:132], gyb[1:31, 2:131], weight), (big.T[:180, :50], gyb.T[:30, :50], weight),
                     (big[:1, :40].expand(180, 40), gyb[:1, :1].expand(30, 40), weight), (big[:180, :64], gyb[:30, :64], mk(g, 6, 30).to(dev).T)):
        want, bound = ref.combine(z.cpu(), w.cpu())
        within(zs.zs_combine(z, w), want, bound(F32), z.stride())
        (gz, gw), (bz, bw) = ref.combine_grads(gy.cpu(), z.cpu(), w.cpu())
        got = zs.zs_combine_backward(gy, z, w)
        within(got[0], gz, bz(F32), "grad_z")
        within(got[1], gw, bw(), "grad_weight")


# ---- autograd, streams, graphs, refusals ------------------------------------------------------------------------

def grads_of(fn, leaves, c):
    out = fn(*leaves)
    return torch.autograd.grad((out.double() * c).sum(), [t for t in leaves if t.requires_grad])


def test_autograd(dev):
    """Gradients against float64 autograd of the definition, and against differences of the kernels' own outputs."""
    say("autograd")
    g = gen(11)
    index = tokens(g, 60, 9).to(dev)
    table, x, w, b = mk(g, 9, 24), mk(g, 60, 24), 1 + 0.2 * mk(g, 24), mk(g, 24)
    z, weight = mk(g, 60, 24), mk(g, 20, 3)
    live = (index >= 0) & (index < 9)

    def lookup(t):
        return torch.where(live.to(t.device)[:, None], t[index.to(t.device).clamp(0, 8)] * 0.7, 0.0)

    def norm(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * w + b
    cases = [("embedding", lambda t: zs.embedding(t, index, 0.7), lookup, (table,)),
             ("layer_norm", zs.layer_norm, norm, (x, w, b)),
             ("combine", zs.combine, lambda z, v: (z.view(20, 3, 24) * v[:, :, None]).sum(1), (z, weight))]
    for name, own, plain, args in cases:
        mine = [t.to(dev).requires_grad_() for t in args]
        theirs = [t.double().requires_grad_() for t in args]
        c = torch.randn(own(*mine).shape, generator=g, dtype=torch.float64)
        got, want = grads_of(own, mine, c.to(dev)), grads_of(plain, theirs, c)
        for i, (a, r) in enumerate(zip(got, want)):
            # sums of at most 60 terms of order one, in fp32
            assert (a.double().cpu() - r).abs().max() <= 200 * 2.0 ** -23 * max(1.0, r.abs().max().item()), (name, i)
            # a central difference of step h along a random direction: its own error is h^2 of a third derivative of
            # order one, and 2^-23 / h of rounding, summed over the outputs
            d = torch.randn(args[i].shape, generator=g)
            h = 2.0 ** -7
            at = lambda s: own(*[t.detach() + s * h * d.to(dev) if j == i else t.detach() for j, t in enumerate(mine)]).double()  # noqa: E731
            slope = ((at(1.0) - at(-1.0)) * c.to(dev)).sum().item() / (2 * h)
            exact = (r * d.double()).sum().item()
            assert abs(slope - exact) <= (h * h + 2.0 ** -22 / h) * 30 * c.norm().item(), (name, i, slope, exact)


def test_autograd_of_one_input(dev):
    say("autograd of some inputs")
    x, w = torch.randn(5, 16, device=dev), torch.ones(16, device=dev)
    wg = w.clone().requires_grad_()
    zs.layer_norm(x, wg).sum().backward()
    assert wg.grad.shape == (16,)
    xg = x.clone().requires_grad_()
    zs.layer_norm(xg, w, w).sum().backward()
    assert xg.grad.shape == (5, 16)
    v = torch.rand(5, 1, device=dev).requires_grad_()
    zs.combine(x, v).sum().backward()   # its gradient is an expanded tensor
    assert torch.allclose(v.grad[:, 0], x.sum(1), atol=1e-5)
    t = torch.randn(4, 16, device=dev).requires_grad_()
    zs.embedding(t, torch.tensor([1, 1, 3], device=dev), groups=zs.sorted_groups(torch.tensor([0, 0, 2, 2, 3], dtype=torch.int32, device=dev))).sum().backward()
    assert torch.equal(t.grad.cpu(), torch.tensor([0.0, 2, 0, 1])[:, None].expand(4, 16))


def run_all(a):
    csr = zs.sorted_groups(a["offsets"])
    return (zs.zs_embedding(a["table"], a["index"], 0.5), zs.zs_embedding_backward(a["gy"], a["index"], 40, 0.5), zs.zs_embedding_backward(a["gy"], a["sorted"], 40, 0.5, csr),
            zs.zs_layer_norm(a["x"], a["w"], a["b"]), *zs.zs_layer_norm_backward(a["gy"], a["x"], a["w"]), zs.zs_combine(a["x"], a["weight"]),
            *zs.zs_combine_backward(a["gy"][:600], a["x"], a["weight"]))


def inputs_of_all(dev, dtype):
    g = gen(21)
    index = tokens(g, 3000, 40)
    s = torch.sort(index.clamp(0, 39))[0]
    a = {"table": mk(g, 40, 136, dtype=dtype), "index": index, "sorted": s, "offsets": sorted_form(s, 40)[1], "gy": mk(g, 3000, 136, dtype=dtype),
         "x": mk(g, 3000, 136, dtype=dtype), "w": mk(g, 136), "b": mk(g, 136), "weight": mk(g, 600, 5)}
    return {k: v.to(dev) for k, v in a.items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_graph_replays(dev, dtype):
    say("graph", dtype)
    a = inputs_of_all(dev, dtype)
    run_all(a)
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run_all(a)
    with torch.cuda.graph(other):
        res2 = run_all(a)
    for i in range(4):
        a["x"].add_(0.25)
        a["gy"].mul_(0.5)
        a["table"].add_(1.0)
        a["index"].copy_(a["index"].roll(1))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        eager = run_all(a)
        for got in (res, res2):
            assert all(torch.equal(x, y) for x, y in zip(eager, got)), i


def test_other_stream(dev):
    say("other stream")
    a = inputs_of_all(dev, F32)
    want = run_all(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_all(a)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_two_streams_at_once(dev):
    """Calls in flight on two streams have workspaces of their own."""
    say("two streams")
    a, b = inputs_of_all(dev, F32), inputs_of_all(dev, BF16)
    want = [run_all(a), run_all(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(run_all(x))
    torch.cuda.synchronize()
    for i in range(2):
        for res in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(want[i], res))


def test_outputs_end_where_they_should(dev):
    """Through the C ABI, with marks before and behind every output."""
    say("marks")
    lib, g = layers.load_layers(), gen(31)

    def marked(n, dtype=F32):
        t = torch.full((n + 128,), 77, dtype=dtype, device=dev)
        return t, t[64:].data_ptr()

    def intact(*ts):
        assert all((t[:64] == 77).all() and (t[-64:] == 77).all() and not (t[64:-64] == 77).any() for t in ts)
    for dtype, code in ((F32, 0), (BF16, 1)):
        for M, c, k in ((37, 33, 3), (70, 64, 2), (5, 1031, 7), (9, 4100, 2)):
            x, gy, w = mk(g, M * k, c, dtype=dtype).to(dev), mk(g, M * k, c, dtype=dtype).to(dev), mk(g, c).to(dev)
            index = torch.randint(0, 50, (M * k,), generator=g).to(dev)
            groups = zs.zs_build_csr(index, 50)
            y, at = marked(M * k * c, dtype)
            assert zs._call(dev, lib.zs_embedding, x.data_ptr(), c, (index % (M * k)).data_ptr(), M * k, M * k, c, 1.0, code, at) == 0
            t, t_at = marked(50 * c, dtype)
            size = lib.zs_embedding_backward_workspace_bytes(M * k, c, code)
            ws2 = torch.full((size + 512,), 77, dtype=torch.uint8, device=dev)
            assert zs._call(dev, lib.zs_embedding_backward, gy.data_ptr(), c, index.data_ptr(), groups.rowptr.data_ptr(), groups.perm.data_ptr(), M * k, 50, c, 1.0, code, t_at, ws2.data_ptr(), size) == 0
            n, n_at = marked(M * c, dtype)
            assert zs._call(dev, lib.zs_layer_norm, x.data_ptr(), c, w.data_ptr(), None, M, c, 1e-5, code, n_at) == 0
            gx, gx_at = marked(M * c, dtype)
            gw, gw_at = marked(c)
            gb, gb_at = marked(c)
            size2 = lib.zs_layer_norm_workspace_bytes(M, c)
            ws3 = torch.full((size2 + 512,), 77, dtype=torch.uint8, device=dev)
            assert zs._call(dev, lib.zs_layer_norm_backward, gy.data_ptr(), c, x.data_ptr(), c, w.data_ptr(), M, c, 1e-5, code, gx_at, gw_at, gb_at, ws3.data_ptr(), size2) == 0
            weight = torch.rand(M, k, generator=g).to(dev)
            s, s_at = marked(M * c, dtype)
            assert zs._call(dev, lib.zs_combine, x.data_ptr(), c, weight.data_ptr(), M, k, c, code, s_at) == 0
            gz, gz_at = marked(M * k * c, dtype)
            gv, gv_at = marked(M * k)
            assert zs._call(dev, lib.zs_combine_backward, gy.data_ptr(), c, x.data_ptr(), c, weight.data_ptr(), M, k, c, code, gz_at, gv_at) == 0
            torch.cuda.synchronize()
            intact(y, t, n, gx, gw, gb, s, gz, gv)
            assert (ws2[size:] == 77).all() and (ws3[size2:] == 77).all()
    for M, n, k in ((37, 20, 3), (70, 256, 8), (5, 1000, 64), (300, 5, 2)):
        r, x = layers._Router(k, 1, 1, 1, 2, 0, 1.0), mk(g, M, n).to(dev)
        w, w_at = marked(M * k)
        e, e_at = marked(M * k, torch.int64)
        assert zs._call(dev, lib.zs_route, x.data_ptr(), n, None, r, M, n, 0, w_at, e_at) == 0
        gx, gx_at = marked(M * n)
        expert = e[64:-64].clone()
        r = layers._Router(k, 0, 1, 1, 2, 0, 1.0)
        assert zs._call(dev, lib.zs_route_backward, torch.ones(M, k, device=dev).data_ptr(), x.data_ptr(), n, expert.data_ptr(), r, M, n, 0, gx_at) == 0
        torch.cuda.synchronize()
        assert (w[:64] == 77).all() and (w[-64:] == 77).all() and (e[:64] == 77).all() and (e[-64:] == 77).all()
        assert not (w[64:-64] == 77).any() and (e[64:-64] < n).all()
        intact(gx)


def test_refusals(dev):
    say("refusals")
    t, idx, w = torch.zeros(6, 8, device=dev), torch.zeros(6, dtype=torch.int64, device=dev), torch.ones(8, device=dev)
    bad_value = [lambda: zs.zs_embedding(t[0], idx), lambda: zs.zs_embedding(t, idx[:, None]), lambda: zs.zs_embedding(t, idx.cpu()), lambda: zs.zs_embedding_backward(t, idx[:5], 6),
                 lambda: zs.zs_embedding_backward(t, idx, 6, groups=zs.zs_build_csr(idx, 5)), lambda: zs.zs_embedding_backward(t, idx, 6, groups=zs.zs_build_csr(idx[:4], 6)),
                 lambda: zs.embedding(t, idx, groups=zs.zs_build_csr(idx, 5)), lambda: zs.zs_layer_norm(t, w[:7]), lambda: zs.zs_layer_norm(t, w, w[:3]), lambda: zs.zs_layer_norm(t.cpu(), w),
                 lambda: zs.zs_layer_norm_backward(t[:3], t, w), lambda: zs.zs_combine(t, torch.ones(6, device=dev)), lambda: zs.zs_combine(t, torch.ones(2, 2, device=dev)),
                 lambda: zs.zs_combine_backward(t[:3], t, torch.ones(2, 3, device=dev)), lambda: zs.zs_combine_backward(t[:2, :7], t, torch.ones(2, 3, device=dev))]
    bad_type = [lambda: zs.zs_embedding(t.half(), idx), lambda: zs.zs_embedding(t, idx.int()), lambda: zs.zs_layer_norm(t.double(), w), lambda: zs.zs_layer_norm(t, w.bfloat16()),
                lambda: zs.zs_layer_norm_backward(t.bfloat16(), t, w), lambda: zs.zs_combine(t, torch.ones(2, 3, device=dev).bfloat16()),
                lambda: zs.zs_combine_backward(t[:2].bfloat16(), t, torch.ones(2, 3, device=dev))]
    bad_size = [lambda: zs.zs_embedding(torch.zeros(2, 8193, device=dev), idx), lambda: zs.zs_embedding(t[:0], idx), lambda: zs.zs_embedding(t[:, :0], idx),
                lambda: zs.zs_layer_norm(torch.zeros(2, 8193, device=dev), torch.ones(8193, device=dev)), lambda: zs.zs_combine(torch.zeros(65, 8, device=dev), torch.ones(1, 65, device=dev)),
                lambda: zs.zs_layer_norm(t, w, eps=0.0), lambda: zs.zs_layer_norm_backward(t, t, w, eps=float("nan"))]
    for kind, calls in ((ValueError, bad_value), (TypeError, bad_type), (zs.ZsError, bad_size)):
        for i, call in enumerate(calls):
            with pytest.raises(kind):
                call()
                pytest.fail(f"{kind.__name__} {i}")


def test_offsets_past_32_bits(dev):
    """Tables, rows and slots behind 2^31 elements."""
    say("wide offsets")
    V, c = (1 << 31) // 8192 + 40, 8192
    table = torch.empty(V, c, dtype=BF16, device=dev)
    table.copy_(torch.arange(V, device=dev)[:, None] % 251)
    index = torch.tensor([0, V - 1, V - 20, 7, V - 41], device=dev)
    assert torch.equal(zs.zs_embedding(table, index), (index % 251)[:, None].expand(5, c).to(BF16))
    y = zs.zs_layer_norm(table[-64:], torch.ones(c, device=dev))
    assert (y == 0).all()
    say("wide offsets: all rows")
    out = zs.zs_embedding(table, torch.arange(V - 1, -1, -1, device=dev))
    assert torch.equal(out[-50:], table[:50].flip(0)) and torch.equal(out[:50], table[-50:].flip(0))
    del out
    say("wide offsets: gradient")
    grad = zs.zs_embedding_backward(table, torch.arange(V - 1, -1, -1, device=dev), V)
    assert torch.equal(grad[-50:], table[:50].flip(0)) and torch.equal(grad[:50], table[-50:].flip(0))
    del grad
    say("wide offsets: norm and sum")
    x = zs.zs_layer_norm_backward(table, table, torch.ones(c, device=dev))
    assert (x[0][-64:] == 0).all() and x[2].eq(x[2][0]).all()
    del x
    M = V // 2
    y = zs.zs_combine(table[:2 * M], torch.tensor([[1.0, 2.0]], device=dev).expand(M, 2).contiguous())
    assert torch.equal(y[-30:], (table[:2 * M].view(M, 2, c)[-30:, 0].float() + 2 * table[:2 * M].view(M, 2, c)[-30:, 1].float()).to(BF16))
    gz, gw = zs.zs_combine_backward(y, table[:2 * M], torch.tensor([[1.0, 0.5]], device=dev).expand(M, 2).contiguous())
    assert torch.equal(gz.view(M, 2, c)[-30:, 0], y[-30:]) and torch.equal(gz.view(M, 2, c)[-30:, 1], y[-30:] / 2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("at", [0, 3, 8])
def test_rows_end_anywhere(dev, dtype, at):
    """Rows that end at every place of a 16-byte chunk, between elements that are not numbers: none of those counts."""
    M, k, V = 61, 3, 19
    for c in (*range(1, 18), *range(260, 269), *range(1017, 1026)):
        say("rows end anywhere", dtype, at, c)
        g = gen(c)

        def among(rows, std=1.0):
            big = torch.full((rows, at + c + 5), float("nan"), dtype=dtype)
            big[:, at:at + c] = mk(g, rows, c, std=std, dtype=dtype)
            return big[:, at:at + c], big.to(dev)[:, at:at + c]

        (table, dtable), (gy, dgy), (z, dz), (gt, dgt) = among(V), among(M), among(M * k), among(M)
        index = tokens(g, M, V)
        want, bound = ref.embedding(table, index, 1.5)
        within(zs.zs_embedding(dtable, index.to(dev), 1.5), want, bound(dtype), "lookup")
        want, bound = ref.embedding_grad(gy, index, V, 1.5)
        within(zs.zs_embedding_backward(dgy, index.to(dev), V, 1.5), want, bound(dtype), "lookup's gradient")
        w, b = 1 + 0.2 * mk(g, c), mk(g, c)
        want, bound = ref.layer_norm(gt, w, b, 1e-5)
        within(zs.zs_layer_norm(dgt, w.to(dev), b.to(dev)), want, bound(dtype), "layer norm")
        for got, want, bound, n in zip(zs.zs_layer_norm_backward(dgy, dgt, w.to(dev)), *ref.layer_norm_grads(gy, gt, w, 1e-5), "xwb"):
            within(got, want, bound(dtype) if n == "x" else bound(), "layer norm's gradient of " + n)
        for slots in (1, 2, 3):
            rows, weight = M * k // slots, mk(g, M * k // slots, slots)
            zz, dzz, t, dt = z[:rows * slots], dz[:rows * slots], *((gy, dgy) if rows <= M else among(rows))
            t, dt = t[:rows], dt[:rows]
            want, bound = ref.combine(zz, weight)
            within(zs.zs_combine(dzz, weight.to(dev)), want, bound(dtype), ("sum", slots))
            (gz, gw), (bz, bw) = ref.combine_grads(t, zz, weight)
            got = zs.zs_combine_backward(dt, dzz, weight.to(dev))
            within(got[0], gz, bz(dtype), ("sum's gradient of rows", slots))
            within(got[1], gw, bw(), ("sum's gradient of weights", slots))
