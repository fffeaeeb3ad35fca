"""AdamW at the ends of fp32's range: second moments below its normal numbers,
decays of a few of its steps."""
import math

import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests.ops_ref import U, gen

pytestmark = pytest.mark.gpu


def fresh(p, g, fp8, **kw):
    """An optimizer of one tensor with zero states, and what it updates."""
    n = p.numel()
    t = dict(p=p.cuda(), g=g.cuda())
    kind = torch.uint8 if fp8 else torch.float32
    t["m"], t["v"] = (torch.zeros(n, dtype=kind, device="cuda") for _ in range(2))
    if fp8:
        t["ms"], t["vs"] = (torch.zeros((n + 255) // 256, device="cuda") for _ in range(2))
    opt = D.AdamW([t["p"]], [t["g"]], [t["m"]], [t["v"]], m_scale=[t["ms"]] if fp8 else None,
                  v_scale=[t["vs"]] if fp8 else None, **kw)
    return opt, t


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("eps", [1e-30, 2.0 ** -126])
def test_adamw_root_of_a_second_moment_below_normal_numbers(eps, fp8):
    """First steps from gradients whose squares are subnormal or nothing.

    A subnormal v is a whole number of 2^-149, off by at most one of them (half
    for the square's rounding, times 1 - beta2; half for its own), and by four
    roundings.  The update lies between those of the v's at both ends; beside it
    m has two roundings, its factors, the denominator, its reciprocal and the
    products no more than twenty."""
    b1, b2 = 0.9, 0.999
    mags = [10.0 ** (-17 - 0.01 * i) for i in range(700)]  # 1e-17 down to 1e-24
    g = torch.tensor([m if i % 3 else -m for i, m in enumerate(mags)], dtype=torch.float32)
    opt, t = fresh(torch.zeros(700), g, fp8, lr=1.0, beta1=b1, beta2=b2, eps=eps)
    D.adamw_step(opt, 1)
    got = t["p"].cpu().double()
    gd = g.double()
    v = (1 - b2) * gd * gd
    ev = 4 * U * v + 2.0 ** -149
    den = lambda x: torch.sqrt(x.clamp(min=0) / (1 - b2)) + eps  # noqa: E731
    least, most = gd.abs() / den(v + ev) * (1 - 22 * U), gd.abs() / den(v - ev) * (1 + 22 * U)
    assert (got.sign() == -gd.sign()).all()
    off = (got.abs() < least) | (got.abs() > most)
    assert not off.any(), (int(off.sum()), float(gd[off][0]), float(got[off][0]), float(least[off][0]), float(most[off][0]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("decay", [4e-8, 1e-7, 3.3e-7, 1e-3])
def test_adamw_decay_is_rounded_once(decay, fp8):
    """Without gradients and moments only the decay is left: the value less it,
    rounded once to fp32 (half a step: U of the value), the decay itself off by
    two roundings."""
    p = torch.randn(3001, generator=gen(50))
    opt, t = fresh(p, torch.zeros(3001), fp8, lr=1e-3, weight_decay=decay * 1e3)
    D.adamw_step(opt, 1)
    want = p.double() * (1 - decay)
    # half a step of the value's power of two
    half = torch.exp2(torch.floor(torch.log2(want.abs())) - 24)
    off = (t["p"].cpu().double() - want).abs()
    assert (off <= half * (1 + 2.0 ** -20) + 2 * U * decay * p.abs()).all(), float((off / half).max())


@pytest.mark.parametrize("g", [torch.float32, torch.bfloat16])
def test_norm_of_more_blocks_than_partial_sums(g):
    """20000 tensors, most of them one block, every seventh two to five: more
    than three times as many blocks as there are partial sums, so a sum takes blocks
    of several tensors and several of one."""
    r = gen(51)
    sizes = [4096 + (i * 977) % 16000 if i % 7 == 3 else (i * 31) % 40 + 1 for i in range(20000)]
    places, at = [], 0
    for n in sizes:
        places.append((at, n))
        at += (n + 3) // 4 * 4  # aligned to 16 bytes here and there only
    x = torch.randn(at, generator=r).to(g)
    used = torch.zeros(at, dtype=torch.bool)
    for a, n in places:
        used[a:a + n] = True
    x[~used] = float("nan")  # between the tensors
    dev = {n: torch.zeros(at, device="cuda") for n in ("p", "m", "v")}
    dev["g"] = x.cuda()
    cut = lambda t: [t[a:a + n] for a, n in places]  # noqa: E731
    opt = D.AdamW(cut(dev["p"]), cut(dev["g"]), cut(dev["m"]), cut(dev["v"]))
    assert opt.desc.run == 4096 and opt.desc.blocks > 3 * 8192
    nb = opt.workspace_bytes()
    ws, out = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda"), torch.zeros(2, device="cuda")
    D.adamw_norm(opt, 1.0, out, ws, nb)
    total = math.sqrt(float(x[used].double().square().sum()))
    norm, scale = out.tolist()
    assert abs(norm - total) <= 2 * U * total and abs(scale - 1 / total) <= 6 * U * scale
