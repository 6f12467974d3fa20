"""The block of experts in the example: its gradients against float64 autograd of the same model in elementary
operations, its run, and one step of it in a captured graph."""
import importlib.util
import os

import pytest
import torch

import edge_node_scatter_amd as zs
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.load()
    spec = importlib.util.spec_from_file_location("train_experts", os.path.join(ROOT, "examples", "train_experts.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain_model(ex, p, f, expert):
    """The example's model in float64 on the CPU from the operators' definitions, its experts given."""
    x = 0.5 * p["table"][f["species"].cpu()] + f["features"].cpu().double()
    d = x - x.mean(1, keepdim=True)
    h = d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * (1 + p["norm"]) + p["shift"]
    s = torch.sigmoid(h @ p["router"][0]).gather(1, expert)
    weight = 1.5 * s / s.sum(1, keepdim=True)
    z = 0
    for j in range(ex.SLOTS):
        up = torch.bmm(h[:, None], p["up"][expert[:, j]])
        z = z + weight[:, j, None] * torch.bmm(torch.nn.functional.silu(up), p["down"][expert[:, j]])[:, 0]
    z = z * (z.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * (1 + p["post"])
    return (x + p["scale"] * z) @ p["readout"]


def test_gradients_of_the_block(example):
    print("[gpu] experts: gradients", flush=True)
    dev = torch.device("cuda:0")
    n = 300
    rows, p = example.make_rows(n, 5, dev), example.make_parameters(6, dev)
    bias = 0.1 * torch.randn(example.EXPERTS, generator=torch.Generator().manual_seed(7)).to(dev)
    out, expert = example.model(p, rows, bias)
    c = torch.randn(n, generator=torch.Generator().manual_seed(0))
    got = torch.autograd.grad((out * c.to(dev)).sum(), list(p.values()))
    p64 = {k: v.detach().cpu().double().requires_grad_() for k, v in p.items()}
    ref_out = plain_model(example, p64, rows, expert.cpu())
    ref = torch.autograd.grad((ref_out * c.double()).sum(), list(p64.values()))
    # a chain of about ten fp32 operators, each within some tens of ulps (2^-23) of its terms' size, through norms
    # whose rows are of ordinary size: 1000 ulps of each array's norm
    tol = 1000 * 2.0 ** -23
    assert (out.double().cpu() - ref_out).norm() <= tol * ref_out.norm()
    for name, g, r in zip(p, got, ref):
        assert (g.double().cpu() - r).norm() <= tol * r.norm(), name
    # the choice: every row in one group of four, its experts the two of largest score and bias there
    q = torch.sigmoid(zs.grouped_mm(zs.layer_norm(0.5 * p["table"][rows["species"]] + rows["features"], 1 + p["norm"], p["shift"]), p["router"], rows["all"]).double()) + bias.double()
    half = q.view(n, 2, 4).sort(2, descending=True)
    group = half[0][:, :, :2].sum(2).argmax(1)
    assert torch.equal(expert, half[1][torch.arange(n, device=dev), group][:, :2] + 4 * group[:, None])


@pytest.mark.parametrize("bits", [32, 8])
def test_training_runs(example, bits):
    print("[gpu] experts: training", bits, flush=True)
    losses = example.train(steps=8, n_rows=500, bits=bits)
    assert len(losses) == 8 and all(0 < v < float("inf") for v in losses)
    assert example.train(steps=8, n_rows=500, bits=bits) == losses


def test_captured_step(example):
    """Products, choice and gradients of a step in a graph, replayed on other inputs."""
    print("[gpu] experts: graph", flush=True)
    dev = torch.device("cuda:0")
    rows = example.make_rows(200, 8, dev)
    bias = torch.zeros(example.EXPERTS, device=dev)
    params = example.make_parameters(9, dev)
    names = list(params)

    def step(t):
        out, expert = example.model(t, rows, bias)
        return (*torch.autograd.grad((out * out).mean(), [t[k] for k in names]), expert)
    static = {k: v.detach().clone().requires_grad_() for k, v in params.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(static)
    for i in range(3):
        with torch.no_grad():
            for k in names:
                static[k].mul_(1.1)
            rows["features"].add_(0.05)
        graph.replay()
        torch.cuda.synchronize()
        # leaves of their own for the eager pass: a graph's leaves stay with the graph
        fresh = {k: static[k].detach().clone().requires_grad_() for k in names}
        for name, a, b in zip(names + ["expert"], step(fresh), res):
            if name == "readout":   # (a library product and its gradient)
                assert torch.allclose(a, b, rtol=1e-4, atol=1e-5)
            else:
                assert torch.allclose(a.double(), b.double(), rtol=1e-3, atol=1e-4), (i, name)
