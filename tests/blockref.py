"""Float64 references of the grouped products, the residual join and AdamW, and the error bounds the tests hold the
kernels to (plain numpy / torch on the CPU, no code shared with the library)."""
import torch

ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half an ulp, relative: 24 and 8 significant bits


def group_rows(offsets, perm, g):
    at = torch.arange(int(offsets[g]), int(offsets[g + 1]))
    return at if perm is None else perm[at].long()


def grouped(x, w, offsets, perm):
    """(y, sum of |products|), float64."""
    x, w = x.double(), w.double()
    y = torch.zeros(x.shape[0], w.shape[2], dtype=torch.float64)
    s = torch.zeros_like(y)
    for g in range(w.shape[0]):
        r = group_rows(offsets, perm, g)
        y[r] = x[r] @ w[g]
        s[r] = x[r].abs() @ w[g].abs()
    return y, s


def grouped_wgrad(x, gy, offsets, perm, n_groups):
    x, gy = x.double(), gy.double()
    out = torch.zeros(n_groups, x.shape[1], gy.shape[1], dtype=torch.float64)
    s = torch.zeros_like(out)
    for g in range(n_groups):
        r = group_rows(offsets, perm, g)
        out[g] = x[r].T @ gy[r]
        s[g] = x[r].abs().T @ gy[r].abs()
    return out, s


def sum_bound(ref, abs_sum, terms, dtype):
    """A sum of `terms` products in fp32, each addition off by at most an fp32 ulp (2^-23) of the running sum of
    magnitudes, rounded once to the output type."""
    inner = (terms + 2) * 2.0 ** -23 * abs_sum
    return inner + ULP[dtype] * (ref.abs() + inner) + 1e-38


def join(x, z, gate, scale, w_post, w_pre, eps):
    x = x.double()
    c = x.shape[1]
    if z is None:
        y = x
    else:
        z = z.double()
        u = z / torch.sqrt((z * z).sum(1, keepdim=True) / c + eps) * w_post.double()
        s = 1.0 if gate is None else torch.sigmoid(gate.double())
        y = x + scale.double() * s * u
    h = None
    if w_pre is not None:
        h = y / torch.sqrt((y * y).sum(1, keepdim=True) / c + eps) * w_pre.double()
    return y, h


def adamw(p, g, m, v, lr, b1, b2, eps, wd, step):
    p, g, m, v = (t.double() for t in (p, g, m, v))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - lr * wd) - lr * (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + eps)
    return p, m, v


def decode(code, top, steps):
    """Values in [0, 1] of 8-bit codes: `steps` codes a power of two, the top code 1, 0 for code 0."""
    down = top - code.long()
    octave = -((down + steps - 1) // steps)
    frac = (-down) % steps
    return torch.where(code > 0, torch.exp2(octave.double()) * (1 + frac.double() / steps), 0.0)
