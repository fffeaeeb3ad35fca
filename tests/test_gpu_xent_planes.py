"""Softmax cross entropy in fp32 of more rows than go through the fp32 instruction
(384): three bfloat16 parts an operand, held to fp32's own rounding."""
import pytest
import torch

from tests import train_ref as R
from tests.ops_ref import U, gen
from tests.test_gpu_xent import check, make, run

pytestmark = pytest.mark.gpu
F64 = torch.float64


# ---------------------------------------------------------------- fp32 in three parts
# Of the six products of the parts, what is not multiplied (mid lo, lo mid, lo lo)
# is below U of the product and the parts add up to the value.  A row's products
# with zeros are exact, so a logit from FEW values of h that are not zero is
# off by 6 FEW additions, each by a step (2 U) of the sum of magnitudes at most.
FEW = 2
PART = (12 * FEW + 2) * U


def sparse(T, d, g, scale=1.0):
    """Rows of `FEW` values that are not zero, anywhere in the row."""
    h = torch.zeros(T, d)
    at = torch.stack([torch.randperm(d, generator=g)[:FEW] for _ in range(T)])
    h.scatter_(1, at, torch.randn(T, FEW, generator=g) * scale)
    return h


def logits_check(h, w, y, scale=1.0, lost=0.0):
    """loss and lse within PART of the magnitudes (and `lost` of each logit)."""
    got = run(h, w, y, scale, grad=False)
    H, W = h.to(F64), w.to(F64)
    z = scale * (H @ W.t())
    # the scale's multiplication, too
    ez = (PART + 3 * U) * abs(scale) * (H.abs() @ W.abs().t()) + lost
    lse = torch.logsumexp(z, 1)
    gap = (z.amax(1) - z.amin(1)).clamp(max=104)
    elo = ez.amax(1) + (2 * gap + 64 + 2 * (w.shape[0] / 32) ** 0.5 + 16) * U + 4 * U * lse.abs()
    R.within(got["lse"], lse, elo, "lse")
    live = (y >= 0) & (y < w.shape[0])
    at = torch.where(live, y, torch.zeros_like(y)).long()[:, None]
    zt, et = z.gather(1, at).squeeze(1), ez.gather(1, at).squeeze(1)
    loss = torch.where(live, lse - zt, torch.zeros((), dtype=F64))
    R.within(got["loss"], loss, elo + et + U * (loss.abs() + zt.abs()), "loss")


@pytest.mark.parametrize("T,V,d", [(385, 3, 256), (513, 129, 512), (700, 1003, 256)])
def test_planes_logits_to_fp32(T, V, d):
    """Logits of tens, so that the target's shows in the loss to fp32's rounding."""
    g = gen(T)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    y[::11] = -100
    logits_check(sparse(T, d, g, 8.0), torch.randn(V, d, generator=g), y)


def test_planes_just_above_a_bfloat16():
    """x = 1 + 2^-7 - 2^-23 in both operands, one word: lse is the product x x.

    To the nearest, x's parts are 1 + 2^-7 and -2^-23.  The first product is exact,
    each of the next two is added with an error of a step (2 U) at most and the
    fourth changes nothing: 4 U.  The exponential's argument is off by half a step
    of 1.44 times the logit, and that is all there is in the logarithm: U of
    the logit.  (Parts by truncation, 1, 2^-7 and so on, leave 7.8 U out.)"""
    T, d = 400, 256
    x = 1 + 2.0 ** -7 - 2.0 ** -23
    h = torch.zeros(T, d)
    h[torch.arange(T), torch.arange(T) % d] = x
    w = torch.full((1, d), x)
    for scale in (1024.0, -1024.0):
        got = run(h, w, torch.zeros(T, dtype=torch.int32), scale, grad=False)
        want = torch.full((T,), scale * x * x, dtype=F64)
        R.within(got["lse"], want, 5 * U * want.abs(), "lse")


@pytest.mark.parametrize("V,T", [(2, 385), (5, 513), (40, 700)])
def test_planes_gradients_to_fp32(V, T):
    """Rows so small that every probability is 1 / V to fp32: dh is a sum over V
    words and dw one over the few rows that have an upstream gradient."""
    d, g = 256, gen(T + V)
    h = torch.randn(T, d, generator=g) * 2.0 ** -24
    w = torch.randn(V, d, generator=g)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    y[5::7] = -100
    dloss = torch.rand(T, generator=g) + 0.5
    counted = torch.zeros(T, dtype=torch.bool)
    counted[3::181] = True
    dloss[~counted] = 0.0
    got = run(h, w, y, 1.0, dloss)
    H, W = h.to(F64), w.to(F64)
    live = y >= 0
    p = torch.softmax(H @ W.t(), 1)
    hot = torch.zeros_like(p)
    hot[live, y[live].long()] = 1.0
    gg = torch.where(live, dloss, torch.zeros(())).to(F64)
    ds = gg[:, None] * (p - hot)
    # logits below 2^-19: their rounding is nothing.  lse has that of the logarithm
    # and its sum, and p = e^-lse two more of lse's size and the exponential's own
    ep = (8 + 8 * torch.log(torch.tensor(float(V))).item()) * U
    # ds: less one and times g, once each; in three parts, none left
    eds = gg[:, None] * (p * ep + 2 * U) + 3 * U * ds.abs()
    Hl = torch.where(live[:, None], H, torch.zeros((), dtype=F64))
    n = int((counted & live).sum())
    for name, ref, mag, err, terms in (("dh", ds @ W, ds.abs() @ W.abs(), eds @ W.abs(), V),
                                       ("dw", ds.t() @ Hl, ds.abs().t() @ Hl.abs(), eds.t() @ Hl.abs(), n)):
        # each additions a step at most, what is left out, and the last factor
        R.within(got[name], ref, err + (12 * terms + 4) * U * mag, name)
    assert (got["dh"][~live] == 0).all()


@pytest.mark.parametrize("T", [385, 513, 700])
@pytest.mark.parametrize("V,d", [(31, 256), (300, 512)])
def test_planes_sizes(T, V, d):
    h, w, y, dloss = make(T, V, d, "f32", seed=11, dead=0.3)
    check(h, w, y, 1.0, dloss, f"{T}x{V}x{d}")


@pytest.mark.parametrize("scale", [0.125, -1.0, 0.0])
def test_planes_scale_and_ones(scale):
    h, w, y, _ = make(400, 150, 256, "f32", seed=12)
    check(h, w, y, scale, None, f"scale {scale}")


def test_planes_large_logits():
    h, w, y, dloss = make(390, 260, 256, "f32", seed=13)
    check(h * 40, w * 8, y, 1.0, dloss, "large logits")


def test_planes_of_small_and_large_values():
    """Weights of 2^-118, whose last part lies below bfloat16's normal numbers:
    what is lost of each value is below 2^-133.  And weights that would round to
    an infinite first part."""
    g = gen(61)
    T, V, d = 400, 70, 256
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    w = torch.randn(V, d, generator=g) * 2.0 ** -118
    # rows of about 2^100 and a scale of 2^20: logits of a few; of each product
    # 2^100 2^20 2^-133 is lost, `FEW` of them, and rows are below 5 2^100
    logits_check(sparse(T, d, g, 2.0 ** 100), w, y, 2.0 ** 20, lost=FEW * 5 * 2.0 ** -13)
    top = torch.finfo(torch.float32).max
    w = torch.where(torch.rand(V, d, generator=g) < 0.5, top, -top)
    logits_check(sparse(T, d, g, 2.0 ** -126), w, y, 1.0, lost=FEW * 5 * 2.0 ** -133 * 2.0 ** 128)
