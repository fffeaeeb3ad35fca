"""Plain 64-bit references and error bounds for the tests of the operators
around the layer (norms, sorted tokens, MXFP4 rows and products).

Bounds count roundings: an fp32 operation is off by at most half a step, 2^-24
of its result, and an output is rounded once to its type (bf16: 2^-9 at most
relative to the value's power of two, taken as finfo.eps / 2 of the value;
fp32: 2^-24).  close() takes the reference, the sum of the magnitudes that
went into each value and the number of fp32 roundings on the longest path."""
from __future__ import annotations

import torch

from bit_quantized_routed_router_amd import ds4moe as D

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DT = {"f32": D.DT_F32, "bf16": D.DT_BF16}
MAGS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def close(got, ref, mag, n, label):
    """|got - ref| <= half a step of got's type at ref + n roundings of mag."""
    half = torch.finfo(got.dtype).eps / 2
    g, r, m = got.detach().cpu().double(), ref.cpu().double(), mag.cpu().double()
    tol = half * r.abs() * (1 + half) + n * U * m * (1 + half) + 1e-38
    same = (g == r) | (g.isnan() & r.isnan())  # equal infinities and NaN on both sides
    bad = ~(((g - r).abs() <= tol) | same)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        at = tuple(i)
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: got {g[at]!r}, "
                             f"reference {r[at]!r}, tolerance {tol[at]!r}")


def rand(g, *shape, kind="f32", scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(TYPES[kind])


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------- sort
def sort_slots(idx, E):
    """counts, offsets, perm, inv by a plain loop over the slots."""
    flat = idx.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for s, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(s)
    counts = [len(v) for v in lists]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    order = [s for v in lists for s in v]
    inv = [-1] * len(flat)
    for p, s in enumerate(order):
        inv[s] = p
    perm = order + [-1] * (len(flat) - len(order))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(counts), i32(offsets), i32(perm), i32(inv).reshape(idx.shape)


# ---------------------------------------------------------------- MXFP4
def mx_quantize(x):
    """(codes int64 [n, cols], scale codes int64 [n, cols / 32]) of fp32 or
    bf16 rows by the format's definition, in 64 bits."""
    n, cols = x.shape
    b = x.double().reshape(n, cols // 32, 32)
    amax = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    safe = torch.where(bad | (amax == 0), torch.ones_like(amax), amax)
    e = torch.frexp(safe).exponent.long() - 1
    sc = (e - 2 + 127).clamp(0, 254)
    r = b.abs() / torch.exp2(sc.double() - 127)[..., None]
    dist = (r[..., None].clamp(max=6.0) - MAGS).abs()
    best = dist.amin(-1, keepdim=True)
    tie = dist == best
    # of two equally near codes the even one
    rank = torch.where(tie, torch.arange(8) % 2, torch.full((), 9))
    code = rank.argmin(-1)
    code = torch.where((b < 0) & (code > 0), code + 8, code)
    code = torch.where((bad | (amax == 0))[..., None], torch.zeros_like(code), code)
    sc = torch.where(bad, torch.full_like(sc, 255), torch.where(amax == 0, torch.zeros_like(sc), sc))
    return code.reshape(n, cols), sc


def mx_pack(code, sc):
    c = code.reshape(-1, 2)
    return torch.cat([(c[:, 0] | (c[:, 1] << 4)).to(torch.uint8), sc.reshape(-1).to(torch.uint8)])


def mx_values(code, sc):
    v = torch.cat([MAGS, -MAGS])[code]
    s = torch.where(sc == 255, torch.full(sc.shape, float("nan"), dtype=torch.float64), torch.exp2(sc.double() - 127))
    return v * s.repeat_interleave(32, dim=1)


def mx_random(g, rows, cols, scale=1.0):
    """A packed random matrix and its values."""
    code, sc = mx_quantize(rand(g, rows, cols, scale=scale))
    return mx_pack(code, sc), mx_values(code, sc)


def random_offsets(g, n, E, tail=0):
    """Ascending offsets of E runs over n - tail rows, empty runs among them."""
    cut = torch.randint(0, n - tail + 1, (max(E - 1, 0),), generator=g).sort().values.tolist()
    return torch.tensor([0] + cut + [n - tail], dtype=torch.int32)
