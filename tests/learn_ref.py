"""The operators that train the token embedding, from their definitions in
64 bits (plain torch on whatever device the inputs are), and the bounds
that their fp32 arithmetic has to keep.

u = 2^-24 is fp32's unit of rounding.  A sum of k terms added in any order is
within (k - 1) u of the sum of the terms' magnitudes; the kernels add at most
`chain` terms one after the other and join the pieces in a tree or in turn,
so `chain` (stated at each use) replaces k.
"""
import torch

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8          # bf16's unit of rounding (8 bits of significand)
F8_MAX = 448.0
SCALE_MIN = 2.0 ** -100


def rms_norm(x, residual, weight, eps):
    h = x.double() + (0.0 if residual is None else residual.double())
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None] * (1.0 if weight is None else weight.double())
    return h, rstd, y


def rms_norm_grad(dy, h, rstd, weight, dsum):
    dy, h, r = dy.double(), h.double(), rstd.double()[:, None]
    g = dy if weight is None else dy * weight.double()
    u = h * r
    dx = r * (g - u * (g * u).mean(1, keepdim=True))
    size = r * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
        size = size + dx.abs()
    return dx, size, (dy * u).sum(0), (dy * u).abs().sum(0)


def embed_grad(dout, ids, is_visual, L, K, V):
    """(level [L, K, D], text [V, D], and the same of |dout|, bad IDs)."""
    d = dout.double()
    vis = torch.ones(ids.shape[0], dtype=torch.bool, device=ids.device) if is_visual is None else is_visual != 0
    out, bad = [], 0
    for x in (d, d.abs()):
        level = torch.zeros((L, K, d.shape[1]), dtype=torch.float64, device=d.device)
        text = torch.zeros((V, d.shape[1]), dtype=torch.float64, device=d.device)
        bad = 0
        for l in range(L):
            ok = vis & (ids[:, l] >= 0) & (ids[:, l] < K)
            bad += int((vis & ~ok).sum())
            level[l].index_add_(0, ids[ok, l].long(), x[ok])
        ok = ~vis & (ids[:, 0] >= 0) & (ids[:, 0] < V)
        if V:
            bad += int((~vis & ~ok).sum())
            text.index_add_(0, ids[ok, 0].long(), x[ok])
        out += [level, text]
    return out[0], out[1], out[2], out[3], bad


def adamw(p, g, m, v, step, lr, betas, eps, decay, factor=1.0):
    p, g, m, v = p.double(), g.double() * factor, m.double(), v.double()
    m = betas[0] * m + (1.0 - betas[0]) * g
    v = betas[1] * v + (1.0 - betas[1]) * g * g
    mh, vh = m / (1.0 - betas[0] ** step), v / (1.0 - betas[1] ** step)
    upd = lr * mh / (vh.sqrt() + eps)
    return p - lr * decay * p - upd, m, v, upd


def f8_step(v):
    """The distance of e4m3 values around v."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30)))
    return torch.pow(2.0, torch.clamp(e, min=-6.0) - 3.0)


def blocks(x, n=256):
    """x [numel] as [blocks, n], zeros after its end."""
    out = torch.zeros(-(-x.numel() // n) * n, dtype=x.dtype, device=x.device)
    out[:x.numel()] = x
    return out.view(-1, n)


def close(got, want, bound, what):
    got, want = got.double(), want.double()
    bound = bound if torch.is_tensor(bound) else torch.as_tensor(bound, dtype=torch.float64, device=want.device)
    off = (got - want).abs()
    bad = ~(off <= bound + 1e-300)
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        o, w = off.expand_as(want).flatten()[i].item(), bound.expand_as(want).flatten()[i].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; element {i}: "
                             f"{got.flatten()[i].item()!r} for {want.flatten()[i].item()!r}, off {o:.3g}, bound {w:.3g}")
