"""GPU parity of the block norms and their gradients (ds4moe_norm_*) with the
formulas in 64 bits.

Roundings on the longest path: a thread adds at most 8 pieces of 8 columns in
a row (64), a wave 6 steps, the waves 8 at most; the root, the mean and the
products around them take less than 16 more, and a gradient adds two such
sums: 100 for a value with one sum, 200 with two.  Sums over T tokens add
T / 512 + 1 terms per team, then 32 partial sums per thread and 16 threads."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests.ops_ref import DT, TYPES, close, gen, rand

pytestmark = pytest.mark.gpu

EPS = 1e-6
GATES = {"none": D.GATE_NONE, "token": D.GATE_TOKEN, "channel": D.GATE_CHANNEL, "full": D.GATE_FULL}


class Case:
    def __init__(self, T, d, h="f32", y="f32", x="f32", gate="none", rho=1.0, weights=True, seed=0):
        g = gen(seed + 131 * T + d)
        self.T, self.d, self.kinds, self.gmode, self.rho = T, d, dict(h=h, y=y, x=x), gate, rho
        self.w = {n: 1 + rand(g, d, scale=0.2) if weights else None for n in ("pre", "post", "next")}
        self.h, self.y = rand(g, T, d, kind=h, scale=2.0), rand(g, T, d, kind=y, scale=0.5)
        self.dh, self.dx = rand(g, T, d, kind=h), rand(g, T, d, kind=x)
        shape = dict(none=None, token=(T,), channel=(d,), full=(T, d))[gate]
        self.gate = None if shape is None else rand(g, *shape)
        self.dev()

    def dev(self):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.norm = D.Norm(self.d, EPS, self.rho, GATES[self.gmode], *(c(self.w[n]) for n in ("pre", "post", "next")))
        self.D = {n: c(getattr(self, n)) for n in ("h", "y", "dh", "dx", "gate")}
        self.ws = self.norm.workspace(self.T)

    def out(self, kind, *shape):
        return torch.full(shape, float("nan"), dtype=TYPES[kind], device="cuda")

    def rows(self, n):
        return self.out(self.kinds[n], self.T, self.d)

    def wt(self, n):
        return torch.ones(self.d, dtype=torch.float64) if self.w[n] is None else self.w[n].double()

    def g64(self):
        g = torch.ones(()) if self.gate is None else self.gate
        g = g.double()
        return g[:, None] if self.gmode == "token" else g

    # ---- calls
    def pre(self):
        x = self.rows("x")
        D.norm_pre(self.norm.desc, self.D["h"], DT[self.kinds["h"]], self.T, x, DT[self.kinds["x"]])
        return x

    def post(self, nxt=True, h_out=None):
        ho = self.rows("h") if h_out is None else h_out
        x = self.rows("x") if nxt else None
        k = self.kinds
        D.norm_post(self.norm.desc, self.D["h"] if h_out is None else h_out, DT[k["h"]], self.D["y"], DT[k["y"]],
                    self.D["gate"], self.T, ho, x, DT[k["x"]])
        return ho, x

    def pre_grad(self, res=True, dw=True):
        dh, w = self.rows("h"), self.out("f32", self.d) if dw else None
        ws = self.ws if dw else (None, 0)
        D.norm_pre_grad(self.norm.desc, self.D["h"], DT[self.kinds["h"]], self.D["dx"], DT[self.kinds["x"]],
                        self.D["dh"] if res else None, self.T, dh, w, *ws)
        return dh, w

    def post_grad(self, dw=True, dg=True):
        dy = self.rows("y")
        w = self.out("f32", self.d) if dw else None
        gg = self.out("f32", *self.gate.shape) if dg and self.gate is not None else None
        D.norm_post_grad(self.norm.desc, self.D["dh"], DT[self.kinds["h"]], self.D["y"], DT[self.kinds["y"]],
                         self.D["gate"], self.T, dy, w, gg, *self.ws)
        return dy, w, gg

    # ---- references: (value, magnitude)
    def ref_pre(self):
        h = self.h.double()
        v = h / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt() * self.wt("pre")
        return v, v.abs()

    def ref_post(self):
        h, y = self.h.double(), self.y.double()
        t = self.g64() * (y / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt() * self.wt("post"))
        ho = self.rho * h + t
        mag = (self.rho * h).abs() + t.abs()
        root = (ho.pow(2).mean(1, keepdim=True) + EPS).sqrt()
        x = ho / root * self.wt("next")
        # the row's error moves its root by at most the errors' mean square
        xm = (mag + ho.abs() * mag.pow(2).mean(1, keepdim=True).sqrt() / root) / root * self.wt("next").abs()
        return (ho, mag), (x, xm)

    def ref_pre_grad(self, res=True):
        h, dx, dh = self.h.double(), self.dx.double(), self.dh.double()
        r = 1 / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt()
        v = dx * self.wt("pre")
        a = self.rho * dh if res else torch.zeros_like(dh)
        out = a + r * (v - h * r * r * (h * v).mean(1, keepdim=True))
        mag = a.abs() + r * (v.abs() + h.abs() * r * r * (h * v).abs().mean(1, keepdim=True))
        t = dx * h * r
        return (out, mag), (t.sum(0), t.abs().sum(0))

    def ref_post_grad(self):
        y, dh, w, g = self.y.double(), self.dh.double(), self.wt("post"), self.g64()
        q = 1 / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt()
        u = dh * g * w
        dy = q * (u - y * q * q * (y * u).mean(1, keepdim=True))
        mag = q * (u.abs() + y.abs() * q * q * (y * u).abs().mean(1, keepdim=True))
        t = dh * g * y * q
        dg = dh * y * q * w
        by = dict(none=lambda v: None, token=lambda v: v.sum(1), channel=lambda v: v.sum(0), full=lambda v: v)[self.gmode]
        return (dy, mag), (t.sum(0), t.abs().sum(0)), (by(dg), by(dg.abs()))

    def check(self, label=""):
        label += f"T={self.T} d={self.d} {self.kinds} gate={self.gmode}"
        over_t = 200 + self.T // 512 + 1 + 48
        close(self.pre(), *self.ref_pre(), 100, label + " x")
        (ho, xn), (rh, rx) = self.post(), self.ref_post()
        close(ho, *rh, 100, label + " h_out")
        close(xn, *rx, 300, label + " x_next")
        for res in (True, False):
            (dh, dw), (rdh, rdw) = self.pre_grad(res), self.ref_pre_grad(res)
            close(dh, *rdh, 200, label + f" dh res={res}")
            close(dw, *rdw, over_t, label + " dw_pre")
        (dy, dw, dg), (rdy, rdw, rdg) = self.post_grad(), self.ref_post_grad()
        close(dy, *rdy, 200, label + " dy")
        close(dw, *rdw, over_t, label + " dw_post")
        if dg is not None:
            close(dg, *rdg, over_t, label + " dgate")


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("h,y,x", [("f32", "f32", "f32"), ("bf16", "f32", "bf16"), ("f32", "bf16", "bf16"),
                                   ("bf16", "bf16", "f32")])
def test_norm_types_and_gates(gate, h, y, x):
    Case(5, 768, h, y, x, gate, rho=0.75).check()


@pytest.mark.parametrize("T,d", [(1, 256), (2, 256), (1, 4096), (3, 2048), (7, 2304), (2, 4352), (3, 8192), (2, 16384),
                                 (513, 256), (1100, 512), (511, 1792), (20001, 256), (257, 12544)])
def test_norm_sizes(T, d):
    Case(T, d, "bf16", "f32", "bf16", "channel" if T % 2 else "token", rho=0.5).check()


def test_norm_without_weights_and_outputs():
    c = Case(9, 512, gate="full", weights=False)
    c.check()
    ref = c.post_grad()
    got = c.post_grad(dw=False)
    assert got[1] is None and torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])
    got = c.post_grad(dg=False)
    assert got[2] is None and torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    c2 = Case(9, 512, gate="channel")
    ref, got = c2.post_grad(), c2.post_grad(dw=False)
    assert torch.equal(got[2], ref[2])
    assert torch.equal(c.pre_grad(dw=False)[0], c.pre_grad()[0])
    assert torch.equal(c.post(nxt=False)[0], c.post()[0])


def test_norm_in_place():
    c = Case(33, 1024, "bf16", "bf16", "bf16", "token")
    ho, x = c.post()
    h2 = c.D["h"].clone()
    got, x2 = c.post(h_out=h2)
    assert got is h2 and torch.equal(h2, ho) and torch.equal(x2, x)
    dh, _ = c.pre_grad()
    buf = c.D["dh"].clone()
    D.norm_pre_grad(c.norm.desc, c.D["h"], D.DT_BF16, c.D["dx"], D.DT_BF16, buf, c.T, buf, None, None, 0)
    assert torch.equal(buf, dh)
    dy, _, _ = c.post_grad()
    buf = c.D["y"].clone()
    D.norm_post_grad(c.norm.desc, c.D["dh"], D.DT_BF16, buf, D.DT_BF16, c.D["gate"], c.T, buf, None, None, None, 0)
    assert torch.equal(buf, dy)


def test_norm_zero_rows_and_stray_values():
    """A row of zeros (a token that no expert took) passes the residual through;
    an infinity or a NaN stays in its row."""
    c = Case(6, 512, gate="token")
    c.y[1] = 0
    c.h[2] = 0
    c.y[3, 17] = float("nan")
    c.h[4, 5] = float("inf")
    c.dev()
    (ho, xn), (rh, rx) = c.post(), c.ref_post()
    assert torch.equal(ho[1].cpu(), c.h[1])
    assert ho[3].isnan().all() and xn[3].isnan().all()
    keep = [0, 1, 2, 5]
    close(ho[keep], rh[0][keep], rh[1][keep], 100, "h_out")
    close(xn[keep], rx[0][keep], rx[1][keep], 300, "x_next")
    x, (rx, mx) = c.pre(), c.ref_pre()
    assert (x[2] == 0).all() and x[4, 5].isnan()
    keep = [0, 1, 2, 3, 5]
    close(x[keep], rx[keep], mx[keep], 100, "x")
    (dy, _, _), (rdy, _, _) = c.post_grad(), c.ref_post_grad()
    keep = [0, 1, 2, 4, 5]
    close(dy[keep], rdy[0][keep], rdy[1][keep], 200, "dy")


def test_norm_small_and_large_magnitudes():
    """Rows near the smallest normal numbers (eps rules) and near 2^55."""
    c = Case(3, 256)
    c.h[0] *= 2.0 ** -60
    c.y[0] *= 2.0 ** -60
    c.h[1] *= 2.0 ** 50
    c.y[1] *= 2.0 ** 50
    c.dev()
    c.check()


def test_norm_gradients_against_differences():
    """The gradients against central differences of the 64-bit forward: the
    loss <h_out, dh> + <x, dx> of the pair of norms moves along random
    directions as the kernels' gradients say (step 1e-4, third-order remainder
    below 1e-6 of the slopes; kernel gradients in fp32: 1e-5)."""
    c = Case(4, 256, gate="channel", rho=0.5)
    g = gen(9)

    def loss():
        (ho, _), _ = c.ref_post()
        x, _ = c.ref_pre()
        return float((ho * c.dh.double()).sum() + (x * c.dx.double()).sum())

    dh, dw_pre = c.pre_grad()
    dy, dw_post, dg = c.post_grad()
    c.h, c.y, c.gate = c.h.double(), c.y.double(), c.gate.double()
    c.w = {n: v.double() for n, v in c.w.items()}
    holders = [(c, "h", dh), (c, "y", dy), (c, "gate", dg), (c.w, "pre", dw_pre), (c.w, "post", dw_post)]
    for holder, name, grad in holders:
        get = (lambda: holder[name]) if isinstance(holder, dict) else (lambda: getattr(holder, name))
        put = (lambda v: holder.__setitem__(name, v)) if isinstance(holder, dict) else (lambda v: setattr(holder, name, v))
        base = get()
        v = torch.randn(base.shape, generator=g, dtype=torch.float64)
        put(base + 1e-4 * v)
        up = loss()
        put(base - 1e-4 * v)
        down = loss()
        put(base)
        want = (up - down) / 2e-4
        prod = grad.cpu().double() * v
        assert abs(float(prod.sum()) - want) <= 1e-5 * float(prod.abs().sum()) + 1e-6 * abs(want), name


def test_norm_repeats_bit_for_bit():
    c = Case(700, 1024, "bf16", "f32", "bf16", "channel")
    a, b = [t for f in (c.pre_grad, c.post_grad) for t in f()], [t for f in (c.pre_grad, c.post_grad) for t in f()]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_norm_on_another_stream():
    c = Case(64, 1024)
    ref = c.pre()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = c.rows("x")
    s.wait_stream(torch.cuda.current_stream())
    D.norm_pre(c.norm.desc, c.D["h"], D.DT_F32, c.T, x, D.DT_F32, s)
    s.synchronize()
    a = x
    assert torch.equal(a, ref)
