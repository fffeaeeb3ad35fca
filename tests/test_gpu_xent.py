"""Softmax cross entropy over a vocabulary and its gradients against the
formulas in 64 bits."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests import train_ref as R
from tests.ops_ref import TYPES, gen

pytestmark = pytest.mark.gpu


def run(h, w, target, scale=1.0, dloss=None, grad=True, want=("dh", "dw")):
    T, d = h.shape
    V = w.shape[0]
    dt = D.DT_F32 if h.dtype == torch.float32 else D.DT_BF16
    hd, wd, td = h.cuda(), w.cuda(), target.cuda()
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    n = D.xent_workspace_bytes(dt, T, V, d, grad)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type
    D.xent(hd, wd, dt, T, V, d, scale, td, loss, lse, ws, n)
    out = dict(loss=loss, lse=lse)
    if grad:
        out["dh"] = torch.full_like(hd, 7.0) if "dh" in want else None
        out["dw"] = torch.full_like(wd, 7.0) if "dw" in want else None
        ws.fill_(0xFF)
        D.xent_grad(hd, wd, dt, T, V, d, scale, td, lse, None if dloss is None else dloss.cuda(), out["dh"], out["dw"],
                    ws, n)
    torch.cuda.synchronize()
    return {k: v if v is None else v.cpu() for k, v in out.items()}


def make(T, V, d, kind, seed=0, dead=0.0, scale=1.0):
    g = gen(seed * 7919 + T * 31 + V)
    h = torch.randn(T, d, generator=g).to(TYPES[kind])
    w = (torch.randn(V, d, generator=g) * 1.5 / (scale * d ** 0.5)).to(TYPES[kind])
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    if dead:
        y[torch.rand(T, generator=g) < dead] = -100
        y[torch.rand(T, generator=g) < dead / 4] = V
    return h, w, y, torch.rand(T, generator=g) + 0.5


def check(h, w, y, scale, dloss, label):
    got = run(h, w, y, scale, dloss)
    ref = R.Xent(h, w, y, scale, dloss)
    R.within(got["lse"], ref.lse, ref.elo, label + " lse")
    R.within(got["loss"], ref.loss, ref.el, label + " loss")
    R.within(got["dh"], ref.dh, ref.edh, label + " dh")
    R.within(got["dw"], ref.dw, ref.edw, label + " dw")
    assert (got["loss"][~ref.live] == 0).all() and (got["dh"][~ref.live] == 0).all()


# rows and words at the borders of fragments, tiles and pieces
SIZES = [(1, 1, 256), (1, 2, 256), (3, 31, 256), (16, 33, 512), (31, 127, 256), (32, 128, 256), (33, 129, 512),
         (64, 64, 256), (65, 200, 256), (127, 256, 768), (128, 257, 256), (129, 1000, 256), (255, 511, 256),
         (300, 300, 512), (2, 5003, 256)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,d", SIZES)
def test_xent_sizes(T, V, d, kind):
    h, w, y, dloss = make(T, V, d, kind, dead=0.3 if T > 2 else 0.0)
    check(h, w, y, 1.0, dloss, f"{T}x{V}x{d} {kind}")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.125, -1.0, 0.0])
def test_xent_scale_and_ones(scale, kind):
    h, w, y, _ = make(40, 150, 256, kind, seed=1)
    check(h, w, y, scale, None, f"scale {scale}")


@pytest.mark.parametrize("kind,T,V,d", [("bf16", 1030, 1500, 256), ("bf16", 520, 4100, 1024), ("f32", 300, 2100, 512),
                                        ("bf16", 40, 6000, 2048)])
def test_xent_large_tiles(kind, T, V, d):
    """Enough blocks for the larger tiles, several parts of dh's sum."""
    h, w, y, dloss = make(T, V, d, kind, seed=2, dead=0.1)
    check(h, w, y, 1.0, dloss, f"{T}x{V}x{d} {kind}")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_xent_without_any_target(kind):
    h, w, y, dloss = make(70, 100, 256, kind, seed=3)
    got = run(h, w, torch.full_like(y, -1), 1.0, dloss)
    assert (got["loss"] == 0).all() and (got["dh"] == 0).all() and (got["dw"] == 0).all()
    assert torch.isfinite(got["lse"]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("want", ["dh", "dw"])
def test_xent_one_gradient(want, kind):
    h, w, y, dloss = make(100, 300, 256, kind, seed=4, dead=0.2)
    both, one = run(h, w, y, 1.0, dloss), run(h, w, y, 1.0, dloss, want=(want,))
    assert torch.equal(one[want], both[want])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_xent_masked_rows_hide_what_they_hold(kind):
    h, w, y, dloss = make(90, 200, 256, kind, seed=5)
    y[::3] = -100
    want = run(h, w, y, 1.0, dloss)
    h2 = h.clone()
    h2[::3] = float("nan")
    h2[3] = float("inf")
    d2 = dloss.clone()
    d2[::3] = float("nan")
    got = run(h2, w, y, 1.0, d2)
    live = y >= 0
    for name in ("dh", "dw", "loss"):
        assert torch.equal(got[name], want[name]), name
    assert torch.equal(got["lse"][live], want["lse"][live])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_xent_non_finite_rows_stay_apart(bad, kind):
    h, w, y, dloss = make(70, 150, 256, kind, seed=6)
    want = run(h, w, y, 1.0, dloss)
    h[5, 7] = bad
    got = run(h, w, y, 1.0, dloss)
    others = torch.arange(70) != 5
    for name in ("loss", "lse", "dh"):
        assert torch.equal(got[name][others], want[name][others]), name
        assert not torch.isfinite(got[name][5]).any(), name


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_xent_large_logits(kind):
    """Logits of hundreds: one word takes all of the probability, the others underflow."""
    h, w, y, dloss = make(33, 260, 256, kind, seed=7)
    check(h * 40, w * 8, y, 1.0, dloss, "large logits")


def test_xent_same_target_and_small_dloss():
    """Every row on one word, and upstream gradients near fp32's smallest."""
    h, w, y, dloss = make(200, 64, 256, "bf16", seed=8)
    y.fill_(63)
    check(h, w, y, 1.0, dloss / 4096, "one word")
    small = run(h, w, y, 1.0, dloss * 2.0 ** -100)
    full = run(h, w, y, 1.0, dloss)
    # a power of two changes no rounding above bf16's normal numbers
    assert torch.equal(small["dw"].double() * 2.0 ** 100, full["dw"].double())


def test_xent_gradient_against_differences():
    """Central differences in 64 bits: off by h^2 / 6 of a third derivative
    below the cube of the weights' size, 1."""
    h, w, y, _ = make(6, 20, 256, "f32", seed=9)
    got = run(h, w, y)

    def total(hh, ww):
        z = hh @ ww.t()
        return (torch.logsumexp(z, 1) - z.gather(1, y.long()[:, None]).squeeze(1)).sum()

    H, W, e = h.double(), w.double(), 1e-4
    for at in ((0, 0), (5, 255), (2, 100)):
        a, b = H.clone(), H.clone()
        a[at] += e
        b[at] -= e
        diff = (total(a, W) - total(b, W)) / (2 * e)
        assert abs(float(diff) - float(got["dh"][at])) <= 1e-5
    for at in ((0, 0), (19, 255), (7, 100)):
        a, b = W.clone(), W.clone()
        a[at] += e
        b[at] -= e
        diff = (total(H, a) - total(H, b)) / (2 * e)
        assert abs(float(diff) - float(got["dw"][at])) <= 1e-5


def test_xent_repeats_bit_for_bit():
    h, w, y, dloss = make(300, 3000, 512, "bf16", seed=10, dead=0.1)
    a = run(h, w, y, 1.0, dloss)
    for _ in range(2):
        b = run(h, w, y, 1.0, dloss)
        assert all(torch.equal(a[k], b[k]) for k in a)
