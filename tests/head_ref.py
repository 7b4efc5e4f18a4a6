"""The operators of a model's head from their definitions in 64 bits (plain torch
on whatever device the inputs are), and the bounds that their fp32 arithmetic
has to keep.

U = 2^-24 is fp32's unit of rounding.  A sum of k terms added in any order is
within (k - 1) U of the sum of the terms' magnitudes; `chain` (stated at each use)
is the longest run of additions that the kernels make one after the other.
"""
import torch

from learn_ref import BF16_HALF, F8_MAX, SCALE_MIN, U

BF16_ROUND = BF16_HALF * (1 + 2 ** -8)


def layer_norm(x, residual, weight, bias, eps):
    h = x.double() + (0.0 if residual is None else residual.double())
    mean = h.mean(1)
    c = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + eps)
    w = 1.0 if weight is None else weight.double()
    y = c * rstd[:, None] * w + (0.0 if bias is None else bias.double())
    return h, mean, rstd, y


def layer_norm_bounds(h, mean, rstd, weight, bias, chain, added):
    """Bounds of (mean, rstd, y) in fp32.  c = h - mean is off by its own rounding and by
    the mean's, (chain) U mean|c|; where a residual was added, h is off by U |h| itself."""
    r = rstd[:, None]
    c = h - mean[:, None]
    w = 1.0 if weight is None else weight.double().abs()
    off = chain * U * (c.abs() + c.abs().mean(1, keepdim=True))
    if added:
        off = off + U * (h.abs() + h.abs().mean(1, keepdim=True))
    rel = 2 * chain * U + off.amax(1, keepdim=True) * r
    b_mean = chain * U * (h - mean[:, None]).abs().mean(1) + 2 * U * mean.abs()
    if added:
        b_mean = b_mean + U * h.abs().mean(1)
    y0 = c.abs() * r * w
    return b_mean, rel[:, 0] * rstd, off * r * w + rel * y0 + 4 * U * (y0 + (0.0 if bias is None else bias.double().abs()))


def layer_norm_grad(dy, h, mean, rstd, weight, dsum):
    dy, r = dy.double(), rstd.double()[:, None]
    u = (h.double() - mean.double()[:, None]) * r
    g = dy if weight is None else dy * weight.double()
    gu = g * u
    dx = r * (g - g.mean(1, keepdim=True) - u * gu.mean(1, keepdim=True))
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + u.abs() * gu.abs().mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
        size = size + dx.abs()
    return dx, size, (dy * u).sum(0), (dy * u).abs().sum(0), dy.sum(0), dy.abs().sum(0)


def block_scale(x, block_rows):
    """Scales of x [rows, cols] in 64 bits: [rows, blocks] or [row blocks, blocks]."""
    r, c = x.shape
    rb, cb = -(-r // block_rows), -(-c // 128)
    p = torch.zeros((rb * block_rows, cb * 128), dtype=torch.float64, device=x.device)
    p[:r, :c] = x.double().abs()
    return (p.view(rb, block_rows, cb, 128).amax((1, 3)) / F8_MAX).clamp(min=SCALE_MIN)


def spread(scale, shape):
    """A scale tensor of any layout, for every element of [rows, k]."""
    rows, k = shape
    s = scale.double()
    if s.dim() == 1:
        return s[:, None].expand(rows, k)
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :k]


def matmul(a, sa, b, sb):
    """(product, product of magnitudes) in 64 bits."""
    x = a.double() * spread(sa, a.shape)
    y = (b.double() * spread(sb, b.shape)).t().contiguous()
    return torch.mm(x, y), torch.mm(x.abs(), y.abs())


def matmul_bound(size, k, eight=False):
    """Products of e4m3 values are exact; 128 of them are added (each addition within
    two units, should the hardware cut off), a block's sum is multiplied by the product of two
    scales (two roundings) and added to the others'.  eight: the matrix cores' 8-bit products,
    as bf16 results may use: eight at a time are added with what lies below 2^-13 of the
    largest cut off, so each of the seven others loses less than that."""
    return (256 + -(-k // 128) + 8) * U * size + (7 * 2.0 ** -13 * size if eight else 0.0)


class Logits:
    """A row's softmax in 64 bits, and how far fp32 may be from it.

    d = (M - x) / T has two roundings and the exponential about one unit, so exp(-d) is
    within (3 d + 4) U of itself, and the sum over all but the largest within
    `chain` U more.  log S is log1p of that sum (two units)."""

    def __init__(self, x, T, chain):
        self.x = x.double()
        self.M = self.x.amax(1, keepdim=True)
        self.d = (self.M - self.x) / T
        e = torch.exp(-self.d)
        first = torch.zeros_like(e).scatter_(1, self.d.argmin(1, keepdim=True), 1.0)
        rest = (e * (1 - first)).sum(1, keepdim=True)
        self.S = 1 + rest
        self.logS = torch.log1p(rest)
        self.p, self.logp = e / self.S, -self.d - self.logS
        pd = torch.where(self.p > 0, self.p * self.d, 0.0)
        self.H = self.logS + pd.sum(1, keepdim=True)
        mass = rest / self.S
        self.b_logS = U * ((chain + 4) * mass + 4 * pd.sum(1, keepdim=True) + 4 * self.logS)
        pdd = torch.where(self.p > 0, self.p * self.d * self.d, 0.0).sum(1, keepdim=True)
        self.b_H = self.b_logS * (1 + self.H) + U * ((chain + 12) * pd.sum(1, keepdim=True) + 6 * pdd + 4 * self.H)
        dd = torch.where(self.d < 1e30, self.d, 0.0)
        self.b_logp = self.b_logS + U * (3 * dd + 2 * torch.where(self.d < 1e30, self.logp.abs(), 0.0))
        self.rel_p = U * (4 * dd + 12) + self.b_logS    # p from the kernel's own statistics


def logprob_grad(r, ids, dlogprob, dentropy, T):
    """(dlogits, bound) in 64 bits for Logits r."""
    n = r.p.shape[0]
    ok = (ids >= 0) & (ids < r.p.shape[1])
    g = torch.zeros((n, 1), dtype=torch.float64, device=r.p.device) if dlogprob is None else \
        torch.where(ok, dlogprob.double(), 0.0)[:, None]
    gh = torch.zeros_like(g) if dentropy is None else dentropy.double()[:, None]
    at = ids.clamp(0, r.p.shape[1] - 1).long()[:, None]
    hot = torch.zeros_like(r.p).scatter_(1, at, ok.double()[:, None])
    lp = torch.where(r.p > 0, r.logp, 0.0)
    one = torch.where(hot > 0, -torch.expm1(r.logp), -r.p)
    dx = (g * one - gh * r.p * (lp + r.H)) / T
    size = g.abs() * (r.p * r.rel_p + 8 * U * one.abs())
    size = size + gh.abs() * r.p * ((lp.abs() + r.H) * (r.rel_p + 8 * U) + 8 * U * (r.H + r.logS) + r.b_H + r.b_logS)
    return dx, size / T


def distill(x, ids, teacher, T, tail, chain):
    """(loss, its bound, dlogits / dloss, its bound) in 64 bits, row by row (small inputs)."""
    n, V = x.shape
    r = Logits(x, T, chain)
    loss, b_loss = (torch.zeros(n, dtype=torch.float64, device=x.device) for _ in range(2))
    dx, b_dx = torch.zeros_like(r.p), torch.zeros_like(r.p)
    for i in range(n):
        seen, entries = set(), []
        for j, t in enumerate(ids[i].tolist()):
            if 0 <= t < V and t not in seen:
                seen.add(t)
                entries.append((j, t))
        if not entries:
            continue
        at = torch.tensor([t for _, t in entries], device=x.device)
        v = teacher[i, torch.tensor([j for j, _ in entries], device=x.device)].double()
        if not tail and bool((v == -torch.inf).all()):
            continue
        logq = v if tail else torch.log_softmax(v / T, 0)
        q = logq.exp()
        has = q > 0
        loss[i] = (q[has] * (logq[has] - r.logp[i, at][has])).sum()
        # S is a plain sum here: chain U of all of it
        b_S = U * (chain + 4 + 4 * float((r.p[i] * torch.where(r.p[i] > 0, r.d[i], 0.0)).sum()))
        b_loss[i] = b_S * (q.sum() + 1e-6)
        p = r.p[i]
        rel = r.rel_p[i] + b_S
        d, b = p.clone(), p * rel
        if tail:
            rest = (1.0 - q.sum()).clamp(min=0.0)
            z = -r.d[i].clone()
            z[at] = -torch.inf
            lt = torch.logsumexp(z, 0)
            if bool(lt > -torch.inf):
                share = torch.exp(z - lt)
                dt = torch.where(share > 0, z.amax() - z, 0.0)
                b_T = U * (chain + 8 + 4 * float((share * dt).sum()))
                if float(rest) > 0:
                    loss[i] += rest * (torch.log(rest) - (lt - r.logS[i, 0]))
                    b_loss[i] += rest * (b_T + b_S)
                d = d - rest * share
                b = b + rest * share * (b_T + U * (4 * dt + 12))
            elif float(rest) > 2.0 ** -16:     # below: the logarithms' rounding
                loss[i] = torch.inf
        d[at] = p[at] - q
        b[at] = p[at] * rel[at] + 2 * U * (p[at] + q)
        b_loss[i] += 2 * U * loss[i].abs().clamp(max=1e30) + 2 * U
        dx[i], b_dx[i] = d / T, (b + 4 * U * d.abs()) / T
    return loss, b_loss, dx, b_dx
