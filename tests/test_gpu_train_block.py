"""The example block: its gradients against float64 autograd of the same model in elementary operations, and training."""
import importlib.util
import os

import pytest
import torch

import blockref
import edge_node_scatter_amd as zs
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.load()
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain_model(p, f, n_nodes):
    """The example's model in float64 on the CPU, from the operators' definitions."""
    C = p["readout"].shape[1]
    groups = lambda csr: torch.repeat_interleave(torch.arange(csr.n_nodes), csr.rowptr.cpu().long().diff())  # noqa: E731

    def grouped(x, w, csr):
        index = torch.empty(x.shape[0], dtype=torch.long)
        index[csr.perm.cpu().long()] = groups(csr)
        return torch.bmm(x[:, None], w[index])[:, 0]
    rms = lambda t, w: t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    radial = grouped(f["basis"].cpu().double(), p["radial"], f["pairs"]).view(-1, 3, C)
    slot = torch.tensor([0] * 3 + [1] * 5 + [2] * 7)
    message = f["coupling"].cpu().double()[:, :, None] * radial[:, slot]
    dst = torch.empty(message.shape[0], dtype=torch.long)
    dst[f["csr"].perm.cpu().long()] = groups(f["csr"])
    rows = torch.zeros(n_nodes, 15, C, dtype=torch.float64).index_add(0, dst, message)
    x = torch.cat([torch.zeros(n_nodes, 1, C, dtype=torch.float64), rows], 1).view(-1, C)
    h = rms(x, 1 + p["w_first"])
    y, h = blockref.join(x, grouped(h, p["mix"], f["rows"]), grouped(h, p["gate"], f["rows"]), p["scale"], 1 + p["w_post"], 1 + p["w_pre"], 1e-6)
    return (h.view(-1, 16, C) * p["readout"]).sum((1, 2))


def test_gradients_of_the_block(example):
    print("[gpu] example gradients", flush=True)
    dev = torch.device("cuda:0")
    n = 40
    frame = example.make_frame(n, 900, 5, dev)
    p = example.make_parameters(6, dev)
    out = example.model(p, frame)
    c = torch.randn(n, generator=torch.Generator().manual_seed(0))
    got = torch.autograd.grad((out * c.to(dev)).sum(), list(p.values()))
    p64 = {k: v.detach().cpu().double().requires_grad_() for k, v in p.items()}
    ref_out = plain_model(p64, frame, n)
    ref = torch.autograd.grad((ref_out * c.double()).sum(), list(p64.values()))
    # a chain of about ten fp32 operators, each within some tens of ulps (2^-23) of its terms' size, through norms
    # whose rows are of ordinary size: 1000 ulps of each array's norm
    tol = 1000 * 2.0 ** -23
    assert (out.double().cpu() - ref_out).norm() <= tol * ref_out.norm()
    for name, g, r in zip(p, got, ref):
        assert (g.double().cpu() - r).norm() <= tol * r.norm(), name


@pytest.mark.parametrize("bits", [32, 8])
def test_training_reduces_the_loss(example, bits):
    print("[gpu] example training", bits, flush=True)
    losses = example.train(steps=60, n_nodes=128, n_edges=6000, bits=bits)
    assert losses[-1] < 0.5 * losses[0]
    assert example.train(steps=5, n_nodes=128, n_edges=6000, bits=bits) == losses[:5]
