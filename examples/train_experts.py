"""A small block of experts, trained end to end on one GPU.

    python examples/train_experts.py [--steps 60] [--rows 4096] [--bits 32]

Every row (an atom or a token) is looked up by its species (embedding), normed (layer_norm), and sent to two of eight
experts (route); its experts' products (grouped_mm over expert_groups of the choice, rows laid out for their experts by
another lookup) are summed by the router's weights (combine) and joined with the residual stream (block_join).  A linear
readout is fitted to the values of a teacher of the same form.  All parameters are stepped by AdamW; the router's bias is
moved towards even loads after each step, outside the gradient.  The data are synthetic.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import edge_node_scatter_amd as zs  # noqa: E402

SPECIES, CHANNELS, HIDDEN, EXPERTS, SLOTS = 40, 64, 96, 8, 2
ROUTER = zs.Router(EXPERTS, SLOTS, score="sigmoid", groups=2, top_groups=1, best=2, scale=1.5)


def make_rows(n_rows: int, seed: int, dev) -> dict:
    """Species, features and the groupings that do not change from step to step."""
    gen = torch.Generator().manual_seed(seed)
    share = 1 / torch.arange(1, SPECIES + 1, dtype=torch.float64)
    species = torch.multinomial(share, n_rows, replacement=True, generator=gen).to(dev)
    features = 0.5 * torch.randn(n_rows, CHANNELS, generator=gen)
    slots = torch.arange(0, n_rows * SLOTS + 1, SLOTS, dtype=torch.int32, device=dev)
    return {"species": species, "features": features.to(dev), "by_species": zs.zs_build_csr(species, SPECIES, order=False),
            "all": zs.sorted_groups(torch.tensor([0, n_rows], dtype=torch.int32, device=dev)),
            "token": torch.arange(n_rows, device=dev).repeat_interleave(SLOTS), "by_token": zs.sorted_groups(slots)}


def make_parameters(seed: int, dev) -> dict:
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s, std: (std * torch.randn(*s, generator=gen)).to(dev).requires_grad_()  # noqa: E731
    C, H = CHANNELS, HIDDEN
    return {"table": normal(SPECIES, C, std=1.0), "norm": normal(C, std=0.1), "shift": normal(C, std=0.1),
            "router": normal(1, C, EXPERTS, std=C ** -0.5), "up": normal(EXPERTS, C, H, std=C ** -0.5),
            "down": normal(EXPERTS, H, C, std=H ** -0.5), "scale": normal(C, std=0.5), "post": normal(C, std=0.1),
            "readout": normal(C, std=0.2)}


def model(p: dict, f: dict, bias: torch.Tensor):
    """(one value for each row, the rows' experts)."""
    x = zs.embedding(p["table"], f["species"], 0.5, f["by_species"]) + f["features"]
    h = zs.layer_norm(x, 1 + p["norm"], p["shift"])
    weight, expert = zs.route(zs.grouped_mm(h, p["router"], f["all"]), ROUTER, bias)
    groups = zs.expert_groups(expert, EXPERTS)
    z = zs.grouped_mm(zs.embedding(h, f["token"], 1.0, f["by_token"]), p["up"], groups)
    z = zs.combine(zs.grouped_mm(torch.nn.functional.silu(z), p["down"], groups), weight)
    y = zs.block_join(x, z, None, p["scale"], 1 + p["post"])
    return y @ p["readout"], expert


def train(steps: int = 60, n_rows: int = 4096, bits: int = 32, lr: float = 0.01, log=None) -> list[float]:
    """Losses of `steps` steps."""
    dev = torch.device("cuda:0")
    rows = make_rows(n_rows, 1, dev)
    bias = torch.zeros(EXPERTS, device=dev)
    with torch.no_grad():
        target = model(make_parameters(2, dev), rows, bias)[0]
    p = make_parameters(3, dev)
    opt = zs.AdamW([t.detach() for t in p.values()], lr=lr, betas=(0.9, 0.99), weight_decay=1e-4, state_bits=bits)
    losses = []
    for step in range(steps):
        out, expert = model(p, rows, bias)
        loss = (out - target).square().mean()
        opt.step([g.contiguous() for g in torch.autograd.grad(loss, list(p.values()))])
        load = torch.bincount(expert.flatten(), minlength=EXPERTS + 1)[:EXPERTS].float()
        bias += 0.01 * torch.sign(load.mean() - load)
        losses.append(loss.item())
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {losses[-1]:.5f}  rows of an expert {int(load.min())} to {int(load.max())}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    train(a.steps, a.rows, a.bits, log=lambda s: print(s, flush=True))
