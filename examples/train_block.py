"""A small learned block around the zonal scatter, trained end to end on one GPU.

    python examples/train_block.py [--steps 60] [--nodes 512] [--edges 40000] [--bits 32]

Every edge carries a radial basis; weights chosen by the species of its two ends turn it into the scatter's radial
features (grouped_mm over zs_build_csr of the pair index), the scatter sums them onto nodes, and one residual block
follows on the rows of the padded node layout: a norm, products with weights and a gate by the node's species, and
the gated join with the norm behind it.  A linear readout is fitted to the values of a teacher of the same form.
All parameters are stepped by AdamW.  The data are synthetic.

It shows the calls together, not a potential: a norm and a gate of each padded row by itself do not keep how the rows
of one degree turn into each other under rotation.  Norm weights are kept as their distance from 1, so that the decay
that all tensors share draws them to 1.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import edge_node_scatter_amd as zs  # noqa: E402

SPECIES, BASIS, CHANNELS = 3, 16, 32


def make_frame(n_nodes: int, n_edges: int, seed: int, dev) -> dict:
    """Edges, species, basis and coupling of one synthetic frame, and the groupings that the block reads."""
    gen = torch.Generator().manual_seed(seed)
    src, dst = (torch.randint(0, n_nodes, (n_edges,), generator=gen) for _ in range(2))
    species = torch.randint(0, SPECIES, (n_nodes,), generator=gen)
    centres = torch.linspace(0.5, 4.0, BASIS)
    distance = 0.5 + 3.5 * torch.rand(n_edges, 1, generator=gen)
    basis = torch.exp(-4 * (distance - centres) ** 2)
    coupling = 2 * torch.rand(n_edges, 15, generator=gen) - 1
    pair = (species[src] * SPECIES + species[dst]).to(dev)
    rows = species.repeat_interleave(16).to(dev)   # the 16 padded rows of a node are of its species
    return {"basis": basis.to(dev), "coupling": coupling.to(dev), "csr": zs.zs_build_csr(dst.to(dev), n_nodes),
            "pairs": zs.zs_build_csr(pair, SPECIES * SPECIES, order=False), "rows": zs.zs_build_csr(rows, SPECIES, order=False)}


def make_parameters(seed: int, dev) -> dict:
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s, std: (std * torch.randn(*s, generator=gen)).to(dev).requires_grad_()  # noqa: E731
    C = CHANNELS
    return {"radial": normal(SPECIES * SPECIES, BASIS, 3 * C, std=BASIS ** -0.5), "mix": normal(SPECIES, C, C, std=C ** -0.5),
            "gate": normal(SPECIES, C, 1, std=C ** -0.5), "scale": normal(C, std=0.5), "w_first": normal(C, std=0.1), "w_post": normal(C, std=0.5),
            "w_pre": normal(C, std=0.5), "readout": normal(16, C, std=0.1)}


def model(p: dict, f: dict) -> torch.Tensor:
    """One value for each node."""
    C = CHANNELS
    radial = zs.grouped_mm(f["basis"], p["radial"], f["pairs"]).view(-1, 3, C)
    x = zs.gie_zonal_scatter(f["coupling"], radial, f["csr"]).view(-1, C)
    h = zs.block_norm(x, 1 + p["w_first"])
    z = zs.grouped_mm(h, p["mix"], f["rows"])
    gate = zs.grouped_mm(h, p["gate"], f["rows"])
    _, h = zs.block_join(x, z, gate, p["scale"], 1 + p["w_post"], 1 + p["w_pre"])
    return (h.view(-1, 16, C) * p["readout"]).sum((1, 2))


def train(steps: int = 60, n_nodes: int = 512, n_edges: int = 40000, bits: int = 32, lr: float = 0.01, log=None) -> list[float]:
    """Losses of `steps` steps."""
    dev = torch.device("cuda:0")
    frame = make_frame(n_nodes, n_edges, 1, dev)
    with torch.no_grad():
        target = model(make_parameters(2, dev), frame)
    p = make_parameters(3, dev)
    opt = zs.AdamW([t.detach() for t in p.values()], lr=lr, betas=(0.9, 0.99), weight_decay=1e-4, state_bits=bits)
    losses = []
    for step in range(steps):
        loss = (model(p, frame) - target).square().mean()
        opt.step([g.contiguous() for g in torch.autograd.grad(loss, list(p.values()))])
        losses.append(loss.item())
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--nodes", type=int, default=512)
    ap.add_argument("--edges", type=int, default=40000)
    ap.add_argument("--bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    train(a.steps, a.nodes, a.edges, a.bits, log=lambda s: print(s, flush=True))
