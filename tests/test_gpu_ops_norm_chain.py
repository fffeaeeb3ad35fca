"""The norm gradients as a block uses them when x_next was used too: the next
pre-norm's gradient (ds4moe_norm_pre_grad on h_out, with the gradient of h_out
as the residual path's), then the post-norm's from what that gives.  Along a
random direction of every input the sum of the kernels' gradients meets the
central difference of the loss <h', A> + <x', B> in 64 bits.

Tolerance: each of the two calls is off by at most 200 roundings of the
magnitudes in its sums (as in the calls' own tests), those of the first pass
through the second, and h_out's own rounding moves the first by less than 10
more: 800 half steps of the magnitudes' sum.  The difference's step of 1e-4
leaves a remainder below 1e-6 of them."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests.ops_ref import U, gen, rand

pytestmark = pytest.mark.gpu

EPS = 1e-6
GATES = {"none": D.GATE_NONE, "token": D.GATE_TOKEN, "channel": D.GATE_CHANNEL, "full": D.GATE_FULL}
F32 = D.DT_F32


def wide(g, mode):
    return g[:, None] if mode == "token" else g


@pytest.mark.parametrize("mode", list(GATES))
@pytest.mark.parametrize("T,d,rho", [(1, 256, 1.0), (7, 1792, 0.5), (301, 512, 1.0), (5, 8448, 0.5)])
def test_gradient_through_h_out_and_x_next(T, d, rho, mode):
    g = gen(T + d)
    shape = dict(none=None, token=(T,), channel=(d,), full=(T, d))[mode]
    v = dict(h=rand(g, T, d, scale=2.0), y=rand(g, T, d, scale=0.5), w=1 + rand(g, d, scale=0.2),
             wn=1 + rand(g, d, scale=0.2))
    if shape:
        v["g"] = rand(g, *shape) + 0.5
    A, B = rand(g, T, d), rand(g, T, d)

    c = {n: t.cuda() for n, t in v.items()}
    norm = D.Norm(d, EPS, rho, GATES[mode], w_post=c["w"], w_next=c["wn"])
    following = D.Norm(d, EPS, 1.0, w_pre=c["wn"])
    new = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    ho, xn, dho, dwn, dy, dw = new(T, d), new(T, d), new(T, d), new(d), new(T, d), new(d)
    dg = new(*shape) if shape else None
    ws = norm.workspace(T)
    D.norm_post(norm.desc, c["h"], F32, c["y"], F32, c.get("g"), T, ho, xn, F32)
    D.norm_pre_grad(following.desc, ho, F32, B.cuda(), F32, A.cuda(), T, dho, dwn, *ws)
    D.norm_post_grad(norm.desc, dho, F32, c["y"], F32, c.get("g"), T, dy, dw, dg, *ws)
    grads = dict(h=rho * dho.cpu().double(), y=dy, w=dw, wn=dwn)
    if shape:
        grads["g"] = dg

    def loss(p):
        y, gate = p["y"], wide(p["g"], mode) if shape else 1.0
        hp = rho * p["h"] + gate * (y / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt() * p["w"])
        x = hp / (hp.pow(2).mean(1, keepdim=True) + EPS).sqrt() * p["wn"]
        return float((hp * A.double()).sum() + (x * B.double()).sum())

    p64 = {n: t.double() for n, t in v.items()}
    # magnitudes of what goes into each gradient
    y, w, wn = p64["y"], p64["w"], p64["wn"]
    gate = wide(p64["g"], mode) if shape else torch.ones(1, 1, dtype=torch.float64)
    q = 1 / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    hp = rho * p64["h"] + gate * (y * q * w)
    r = 1 / (hp.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    dx = B.double().abs() * wn
    m = A.double().abs() + r * (dx + hp.abs() * r * r * (hp.abs() * dx).mean(1, keepdim=True))
    u = m * gate.abs() * w
    mg = m * y.abs() * q * w
    mags = dict(h=rho * m, y=q * (u + y.abs() * q * q * (y.abs() * u).mean(1, keepdim=True)),
                w=(m * gate.abs() * y.abs() * q).sum(0), wn=(B.double() * hp * r).abs().sum(0))
    if shape:
        mags["g"] = dict(token=mg.sum(1), channel=mg.sum(0), full=mg)[mode]
    for only in [list(v)] + [[n] for n in v]:
        way = {n: torch.randn(t.shape, generator=g, dtype=torch.float64) if n in only else torch.zeros(t.shape).double()
               for n, t in v.items()}
        step = {s: loss({n: p64[n] + s * 1e-4 * way[n] for n in v}) for s in (1, -1)}
        want = (step[1] - step[-1]) / 2e-4
        got = sum(float((grads[n].cpu().double() * way[n]).sum()) for n in v)
        mag = sum(float((mags[n] * way[n].abs()).sum()) for n in v)
        assert abs(got - want) <= (800 * U + 1e-6) * mag, (only, got, want, mag)
