"""Plain 64-bit references and error bounds for the tests of a training step's
operators (balance loss, cross entropy, AdamW), on the CPU.

Bounds count roundings as ops_ref does: U = 2^-24 for an fp32 operation, half
a step of its type for an output.  An exponential is off by |x| U for its
argument's scaling and 2 U of its own, and adds its argument's error."""
from __future__ import annotations

import torch

from tests.ops_ref import U

F64 = torch.float64


# ---------------------------------------------------------------- balance
def balance(z, idx, off, k):
    """counts, tokens, loss, and p, live, sequence of each token (-1: none)."""
    T, E = z.shape
    B = len(off) - 1
    zz = z.to(F64)
    top = zz.amax(1, keepdim=True)
    e = torch.exp(zz - torch.where(top == -torch.inf, torch.zeros_like(top), top))
    s = e.sum(1, keepdim=True)
    p = torch.where(s == 0, torch.zeros_like(e), e / s)
    on = (idx >= 0) & (idx < E)
    live = on.any(1)
    counts = torch.zeros(B, E, dtype=torch.int32)
    tokens = torch.zeros(B, dtype=torch.int32)
    loss = torch.zeros(B, dtype=F64)
    seq = torch.full((T,), -1)
    for b in range(B):
        lo, hi = max(0, min(T, int(off[b]))), max(0, min(T, int(off[b + 1])))
        mass = torch.zeros(E, dtype=F64)
        for t in range(lo, hi):
            seq[t] = b
            if not live[t]:
                continue
            tokens[b] += 1
            mass += p[t]
            for j in range(idx.shape[1]):
                if on[t, j]:
                    counts[b, idx[t, j]] += 1
        n = int(tokens[b])
        if n:
            loss[b] = E / (k * n * n) * (counts[b].to(F64) * mass).sum()
    return counts, tokens, loss, p, live, seq


def balance_grad(z, idx, off, k, dloss, dslots):
    """dlogits and the magnitudes that its error is counted from: of the
    probability times the counts (about their mean), and of the slots."""
    T, E = z.shape
    counts, tokens, _, p, live, seq = balance(z, idx, off, k)
    d = torch.zeros(T, E, dtype=F64)
    mag = torch.zeros(T, E, dtype=F64)
    for t in range(T):
        b = int(seq[t])
        if b >= 0 and live[t]:
            n = int(tokens[b])
            f = (1.0 if dloss is None else float(dloss[b])) * E / (k * n * n)
            c = counts[b].to(F64) - k * n // E
            d[t] = f * p[t] * (c - (p[t] * c).sum())
            mag[t] = abs(f) * p[t] * (c.abs() + (p[t] * c.abs()).sum())
        if dslots is not None:
            for j in range(idx.shape[1]):
                e = int(idx[t, j])
                if 0 <= e < E:
                    d[t, e] += float(dslots[t, j])
                    mag[t, e] += abs(float(dslots[t, j]))
    return d, mag


def spread(z):
    """The largest |z - max| whose exponential is not nothing in fp32."""
    zz = z.to(F64)
    gap = (zz.amax(1, keepdim=True) - zz).nan_to_num(0.0, 0.0, 0.0)
    return float(gap[gap < 104].max())


# ---------------------------------------------------------------- cross entropy
class Xent:
    """loss, lse, dh, dw in 64 bits with the error that each may have.

    z: products are exact (bf16) or off by 5 U (fp32: the parts that are not
    multiplied, and what three parts leave), and d of them, or 6 d, are added:
    each addition rounds at most at the sum of the magnitudes."""

    def __init__(self, h, w, target, scale, dloss):
        f32 = h.dtype == torch.float32
        d, V = h.shape[1], w.shape[0]
        H, W = h.to(F64), w.to(F64)
        z = scale * (H @ W.t())
        ez = ((6 * d + 5 if f32 else d) + 2) * U * abs(scale) * (H.abs() @ W.abs().t())
        self.lse = torch.logsumexp(z, 1)
        live = (target >= 0) & (target < V)
        y = torch.where(live, target, torch.zeros_like(target)).long()[:, None]
        # 64 sums in a tile, then of the tiles: V is far above both
        gap = (z.amax(1) - z.amin(1)).clamp(max=104)
        self.elo = ez.amax(1) + (2 * gap + 64 + 2 * (V / 32) ** 0.5 + 16) * U + 4 * U * self.lse.abs()
        zt = z.gather(1, y).squeeze(1)
        zero = torch.zeros((), dtype=F64)
        self.loss = torch.where(live, self.lse - zt, zero)
        self.el = self.elo + ez.gather(1, y).squeeze(1) + U * (self.loss.abs() + zt.abs())
        g = torch.where(live, torch.ones_like(self.lse) if dloss is None else dloss.to(F64), zero) * scale
        p = torch.exp(z - self.lse[:, None])
        hot = torch.zeros_like(p).scatter_(1, y, 1.0)
        ds = g[:, None] * (p - hot)
        # ds is taken from the lse that the forward pass gave, and rounded to bf16 (or three parts)
        part = 2.0 ** -8 if not f32 else 2.0 ** -23
        eds = g.abs()[:, None] * (p * (ez + self.elo[:, None] + (z - self.lse[:, None]).abs() * U + 6 * U) + 2 * U * hot)
        eds = eds * (1 + part) + (part + 4 * U) * ds.abs()
        # an exponential below fp32's normal numbers (2^-126) is zero, and so is
        # a ds, held over the largest |g|, below bf16's, which are the same
        eds = eds + (g.abs()[:, None] + g.abs().max()) * 2.0 ** -126
        live_h = torch.where(live[:, None], H, zero)
        n = live.sum().item()
        more = 6 if f32 else 1
        self.dh, self.dw = ds @ W, ds.t() @ live_h
        self.edh = eds @ W.abs() + (more * V + 16) * U * (ds.abs() @ W.abs())
        self.edw = eds.t() @ live_h.abs() + (more * n + 8) * U * (ds.abs().t() @ live_h.abs())
        self.live = live


def within(got, ref, err, label):
    """|got - ref| <= half a step of got's type + err (twice: bounds multiply, and their products are small)."""
    half = torch.finfo(got.dtype).eps / 2
    g, r, e = got.detach().cpu().double(), ref.double(), err.double()
    tol = half * r.abs() * (1 + half) + e * (1 + 2 * half) + 1e-37
    bad = ~((g - r).abs() <= tol)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} values off, first at {at}: got {g[at]!r}, "
                             f"reference {r[at]!r}, tolerance {tol[at]!r}")


# ---------------------------------------------------------------- AdamW
def adamw(p, g, m, v, *, lr, b1, b2, eps, wd, step, s=1.0):
    """New p, m, v in 64 bits and their error bounds (fp32 steps: m and v three
    roundings and those of their factors; the root, the reciprocal and what
    multiplies them eight more)."""
    p, g, m, v = (t.to(F64) for t in (p, g, m, v))
    d = s * g
    m2 = b1 * m + (1 - b1) * d
    v2 = b2 * v + (1 - b2) * d * d
    em = 5 * U * ((b1 * m).abs() + ((1 - b1) * d).abs())
    ev = 6 * U * v2
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    den = torch.sqrt(v2 / c2) + eps
    p2 = p - lr * (wd * p + m2 / c1 / den)
    ep = 3 * U * p.abs() + lr / c1 / den * (em + 16 * U * m2.abs())
    # fp32's smallest numbers: a square below them counts as nothing
    tiny = 2.0 ** -126
    return p2, m2, v2, ep + 4 * U * p2.abs(), em + tiny, ev + tiny
