"""AdamW over many tensors and the norm of their gradients against the
formulas in 64 bits."""
import math

import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests import train_ref as R
from tests.ops_ref import TYPES, U, gen

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
HYPER = dict(lr=2e-3, b1=0.9, b2=0.999, eps=1e-8)


def values(q, scale):
    n = q.numel()
    return q.float().double() * scale.double().repeat_interleave(256)[:n]


def make(sizes, p="f32", g="f32", fp8=False, master=False, seed=0, shift=0):
    """Host tensors of each size; `shift` values before each, so that no vector load fits."""
    r = gen(seed)
    out = []
    for n in sizes:
        row = torch.exp(torch.randn((n + 255) // 256, 1, generator=r)).expand(-1, 256).reshape(-1)[:n]
        t = dict(w=torch.randn(n, generator=r) * 0.1, g=(torch.randn(n, generator=r) * row).to(TYPES[g]))
        t["p"] = t["w"].to(TYPES[p])
        m, v = torch.randn(n, generator=r) * row, torch.rand(n, generator=r) * row * row
        if fp8:
            for name, x in (("m", m), ("v", v.sqrt())):
                b = torch.nn.functional.pad(x, (0, -n % 256)).reshape(-1, 256)
                s = b.abs().amax(1) / 448
                t[name + "s"] = s
                t[name] = (b / torch.where(s > 0, s, torch.ones_like(s))[:, None]).reshape(-1)[:n].to(FP8)
        else:
            t["m"], t["v"] = m, v
        if master:
            t["master"] = t["w"]
        out.append(t)
    return out


def put(x, shift):
    """On the GPU, `shift` values into a buffer of its own, with values around it that must stay."""
    buf = torch.full((x.numel() + 2 * 16 + shift,), 3.0, device="cuda").to(x.dtype)
    a = buf[16 + shift:16 + shift + x.numel()]
    a.copy_(x.cuda())
    return a, buf


def step(ts, wd=0.1, at=7, scale=None, shift=0, hyper=HYPER, stream=None, **kw):
    names = [n for n in ("p", "g", "m", "v", "ms", "vs", "master") if n in ts[0]]
    dev, bufs = {}, []
    for n in names:
        pairs = [put(t[n], shift) for t in ts]
        dev[n] = [a for a, _ in pairs]
        bufs += [(b, a.numel(), shift) for a, b in pairs]
    opt = D.AdamW(dev["p"], dev["g"], dev["m"], dev["v"], m_scale=dev.get("ms"), v_scale=dev.get("vs"),
                  master=dev.get("master"), lr=hyper["lr"], beta1=hyper["b1"], beta2=hyper["b2"], eps=hyper["eps"],
                  weight_decay=wd, **kw)
    s = None if scale is None else torch.tensor([scale], device="cuda")
    D.adamw_step(opt, at, s)
    torch.cuda.synchronize()
    for b, n, sh in bufs:
        head, tail = b[:16 + sh].float(), b[16 + sh + n:].float()
        assert (head == 3).all() and (tail == 3).all(), "values beside a tensor changed"
    return [{n: dev[n][i].cpu() for n in names} for i in range(len(ts))]


def check(ts, got, wd=0.1, at=7, scale=1.0, hyper=HYPER, label=""):
    for i, (t, o) in enumerate(zip(ts, got)):
        name = f"{label} tensor {i}"
        fp8 = "ms" in t
        m = values(t["m"], t["ms"]) if fp8 else t["m"]
        v = values(t["v"], t["vs"]) ** 2 if fp8 else t["v"]
        w = t.get("master", t["p"])
        p2, m2, v2, ep, em, ev = R.adamw(w, t["g"], m, v, wd=wd if isinstance(wd, float) else wd[i], step=at, s=scale, **hyper)
        if fp8:  # a code's value times its scale, and the root's square, are rounded before they are used
            em, ev = em + U * m.abs(), ev + 4 * U * v
            c1, c2 = 1 - hyper["b1"] ** at, 1 - hyper["b2"] ** at
            ep = ep + hyper["lr"] / c1 / (torch.sqrt(v2 / c2) + hyper["eps"]) * (em + 4 * U * m2.abs())
        R.within(o["p"], p2, ep, name + " p")
        if "master" in t:
            R.within(o["master"], p2, ep, name + " master")
            assert torch.equal(o["p"], o["master"].to(o["p"].dtype)), name
        assert torch.equal(o["g"], t["g"])
        if not fp8:
            R.within(o["m"], m2, em, name + " m")
            R.within(o["v"], v2, ev, name + " v")
            continue
        for q, s, want, err, root in (("m", "ms", m2, em, False), ("v", "vs", torch.sqrt(v2), torch.sqrt(v2) * 8 * U, True)):
            n = want.numel()
            b = torch.nn.functional.pad(want.abs(), (0, -n % 256)).reshape(-1, 256)
            top = b.amax(1)
            e = torch.nn.functional.pad(err, (0, -n % 256)).reshape(-1, 256).amax(1)
            assert ((o[s].double() - top / 448).abs() <= (e + 4 * U * top) / 448 + 2.0 ** -126).all(), name + s
            scale_at = o[s].double().repeat_interleave(256)[:n]
            # nearest code: half a step, 2^-4 of the value or 2^-10 of the scale; next to a border either side
            tol = torch.maximum(want.abs() * 2.0 ** -4, scale_at * 2.0 ** -10) * (1 + 2.0 ** -18) + 2 * err + 2.0 ** -126
            val = o[q].float().double() * scale_at
            off = (val - want).abs()
            if root:
                low = (want > 0) & (scale_at > 0)
                assert (o[q].float()[low] > 0).all(), name + " a positive root became 0"
                tol = torch.where(want < scale_at * 2.0 ** -9, scale_at * 2.0 ** -9, tol)
            assert (off <= tol).all(), f"{name} {q}: {float((off - tol).max())} over, of {float(top.max())}"


SIZES = [[1], [7, 8, 9], [255, 256, 257, 1], [4096, 4097, 31], [12345, 3, 511, 8192, 100], [0, 5, 0, 300]]


@pytest.mark.parametrize("p,master", [("f32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_adamw_types_and_sizes(p, g, fp8, master, shift):
    for i, sizes in enumerate(SIZES):
        ts = make(sizes, p, g, fp8, master, seed=i)
        check(ts, step(ts, shift=shift), label=f"{sizes}")


@pytest.mark.parametrize("fp8", [False, True])
def test_adamw_many_tensors(fp8):
    """More than one launch takes, with a decay each."""
    sizes = [(37 * i * i) % 900 + 1 for i in range(150)]
    wd = [0.01 * (i % 5) for i in range(150)]
    ts = make(sizes, "bf16", "f32", fp8, seed=20)
    check(ts, step(ts, wd=wd), wd=wd, label="many")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("at,hyper", [(1, HYPER), (100000, HYPER), (3, dict(lr=1.0, b1=0.0, b2=0.0, eps=1e-3)),
                                      (2, dict(lr=0.0, b1=0.5, b2=0.9, eps=1e-8))])
def test_adamw_steps_and_constants(at, hyper, fp8):
    ts = make([1000, 77], "f32", "f32", fp8, seed=21)
    check(ts, step(ts, at=at, hyper=hyper), at=at, hyper=hyper, label=f"step {at} {hyper}")


def test_adamw_from_nothing():
    """The first step: zero states, zero gradients among them."""
    ts = make([700], "f32", "f32", True, seed=22)
    t = ts[0]
    for n in ("m", "v", "ms", "vs"):
        t[n] = torch.zeros_like(t[n].float()).to(t[n].dtype)
    t["g"][256:512] = 0
    got = step(ts, at=1)
    check(ts, got, at=1, label="first")
    o = got[0]
    assert o["ms"][1] == 0 and o["vs"][1] == 0 and (o["m"].float()[256:512] == 0).all()


def test_adamw_learning_rate_and_step_on_the_device():
    lr, at = torch.tensor([5e-4], device="cuda"), torch.tensor([11], dtype=torch.int32, device="cuda")
    ts = make([513, 20], "f32", "bf16", seed=23)
    got = step(ts, at=0, hyper=dict(HYPER, lr=9.0), lr_dev=lr, step_dev=at)
    check(ts, got, at=11, hyper=dict(HYPER, lr=float(lr)), label="device")


@pytest.mark.parametrize("fp8", [False, True])
def test_adamw_scaled_and_left_out(fp8):
    ts = make([300, 2000], "bf16", "f32", fp8, True, seed=24)
    check(ts, step(ts, scale=0.25), scale=0.25, label="scaled")
    for s in (float("nan"), float("inf"), -float("inf")):
        for t, o in zip(ts, step(ts, scale=s)):
            for n in o:
                assert torch.equal(o[n].view(torch.uint8), t[n].view(torch.uint8)), (s, n)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_adamw_non_finite_gradient_stays_in_its_value_or_block(fp8, bad):
    ts = make([1000], "f32", "f32", fp8, seed=25)
    want = step(ts)[0]
    ts[0]["g"][300] = bad
    got = step(ts)[0]
    one = torch.arange(1000) == 300
    assert torch.equal(got["p"][~one], want["p"][~one])
    if fp8:
        assert got["ms"].isnan().tolist() == [False, True, False, False] == got["vs"].isnan().tolist()
        for n in ("m", "v"):
            keep = torch.arange(1000) // 256 != 1
            assert torch.equal(got[n].view(torch.uint8)[keep], want[n].view(torch.uint8)[keep])
    else:
        assert torch.equal(got["m"][~one], want["m"][~one]) and not torch.isfinite(got["m"][300])


def test_adamw_eight_bits_follow_what_decays():
    """With no gradient the scales fall with every step, and the codes with
    them: after n steps the values are beta^n of the first, to the codes' half
    step and the rounding of each scale."""
    ts = make([512], "f32", "f32", True, seed=26)
    start = values(ts[0]["v"], ts[0]["vs"])
    ts[0]["g"].zero_()
    dev = {n: [ts[0][n].cuda()] for n in ts[0]}
    opt = D.AdamW(dev["p"], dev["g"], dev["m"], dev["v"], m_scale=dev["ms"], v_scale=dev["vs"], beta1=0.9, beta2=0.99)
    for i in range(50):
        D.adamw_step(opt, i + 1)
    got = values(dev["v"][0].cpu(), dev["vs"][0].cpu())
    assert torch.allclose(got, start * 0.99 ** 25, rtol=50 * 4 * U, atol=0)


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 16384], [16385, 7], [(i * 53) % 700 + 1 for i in range(130)], [300001]])
def test_norm(sizes, g, shift):
    ts = make(sizes, "f32", g, seed=30)
    total = math.sqrt(sum(float(t["g"].double().square().sum()) for t in ts))
    grads = [put(t["g"], shift)[0] for t in ts]
    p, m, v = ([torch.zeros(n, device="cuda") for n in sizes] for _ in range(3))
    opt = D.AdamW(p, grads, m, v)
    n = opt.workspace_bytes()
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for most in (total * 0.5, total * 2, float("inf"), 1e-30):
        out = torch.zeros(2, device="cuda")
        D.adamw_norm(opt, most, out, ws, n)
        norm, s = out.tolist()
        assert abs(norm - total) <= 2 * U * total
        # max_norm as an fp32, the quotient rounded once
        assert abs(s - min(1.0, most / total)) <= 6 * U * s


def test_norm_of_large_small_and_no_gradients():
    def norm(*gs):
        gs = [torch.tensor(g, device="cuda") for g in gs]
        p, m, v = ([torch.zeros_like(g) for g in gs] for _ in range(3))
        opt = D.AdamW(p, gs, m, v)
        n = opt.workspace_bytes()
        out = torch.zeros(2, device="cuda")
        D.adamw_norm(opt, 1.0, out, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
        return out.tolist()

    assert norm() == [0.0, 1.0] and norm([0.0, 0.0]) == [0.0, 1.0]
    a = norm([3e30], [4e30])  # squares beyond fp32
    assert abs(a[0] - 5e30) <= 1e24 and abs(a[1] - 2e-31) <= 1e-37
    b = norm([3e-30, 4e-30])  # squares below it
    assert abs(b[0] - 5e-30) <= 1e-36 and b[1] == 1.0
    for bad in (float("nan"), float("inf")):
        n, s = norm([1.0], [2.0, bad])
        assert not math.isfinite(n) and math.isnan(s)


@pytest.mark.parametrize("fp8", [False, True])
def test_adamw_lowest_eps_leaves_values_without_gradients(fp8):
    """The smallest eps: values without gradient and moments only decay, exactly."""
    ts = make([517], fp8=fp8, seed=3)
    for name in ("g", "m", "v"):
        ts[0][name] = torch.zeros_like(ts[0][name].float()).to(ts[0][name].dtype)
    o = step(ts, wd=0.5, hyper=dict(HYPER, lr=1.0, eps=2.0 ** -126))[0]
    assert torch.equal(o["p"], ts[0]["p"] * 0.5) and not o["m"].float().any() and not o["v"].float().any()


def test_adamw_other_gradients_reach_a_captured_step():
    """set_grads writes the table in its place: a graph captured before takes
    the new gradients, and a refused list leaves the old ones."""
    ts = make([300, 4097], seed=8)
    on = {n: [t[n].cuda() for t in ts] for n in ("p", "g", "m", "v")}
    start = {n: [x.clone() for x in on[n]] for n in ("p", "m", "v")}
    opt = D.AdamW(on["p"], on["g"], on["m"], on["v"], lr=HYPER["lr"], beta1=HYPER["b1"], beta2=HYPER["b2"],
                  eps=HYPER["eps"], weight_decay=0.1)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        D.adamw_step(opt, 7)

    def replayed():
        for n, xs in start.items():
            for a, b in zip(on[n], xs):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        return [dict({n: on[n][i].cpu() for n in ("p", "m", "v")}, g=opt.tensors["grad"][i].cpu()) for i in range(2)]

    at = opt.table.data_ptr()
    check(ts, replayed())
    for bad in (on["g"][:1], [g.bfloat16() for g in on["g"]], [on["g"][0], on["g"][1][:-1]], [on["p"][0], on["g"][1]]):
        with pytest.raises((ValueError, D.Ds4moeError)):
            opt.set_grads(bad)
    check(ts, replayed())
    for t in ts:
        t["g"] = -2 * t["g"]
    opt.set_grads([t["g"].cuda() for t in ts])
    assert opt.table.data_ptr() == at
    check(ts, replayed())
    check(ts, replayed())


def test_adamw_past_32_bits():
    """A tensor of more than 2^32 values, bf16 with 8-bit states: its end and a place beyond 2^32 bytes of each."""
    n = (1 << 32) + 70001
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros((n + 255) // 256, device="cuda") for _ in range(2))
    places = [0, (1 << 31) + 12345, (1 << 32) + 3, n - 1]
    for i, a in enumerate(places):
        g[a] = i + 1
    opt = D.AdamW([p], [g], [m], [v], m_scale=[ms], v_scale=[vs], lr=1.0, beta1=0.5, beta2=0.5, eps=1e-8)
    out, nb = torch.zeros(2, device="cuda"), opt.workspace_bytes()
    D.adamw_norm(opt, 100.0, out, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    D.adamw_step(opt, 1, out[1:])
    assert abs(float(out[0]) - math.sqrt(30)) < 1e-6 and float(out[1]) == 1.0
    for i, a in enumerate(places):
        assert float(p[a]) == -1.0 and abs(float(ms[a // 256]) - (i + 1) / 2 / 448) < 1e-7, a
    assert int((p != 0).sum()) == len(places) and int((vs != 0).sum()) == len(places)


@pytest.mark.parametrize("scale", [None, 0.37])
def test_adamw_codes_are_those_of_ieee_operations(scale):
    """States in 8 bits bit for bit: products, sums, root and quotient each
    rounded on the host as on the GPU, two steps in a row."""
    n = 1 << 18
    ts = make([n], "f32", "f32", True, seed=40)
    t = ts[0]
    for at in (5, 6):
        o = step(ts, at=at, scale=scale)[0]
        f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
        d = t["g"] * f(1.0 if scale is None else scale)
        m = t["m"].float() * t["ms"].repeat_interleave(256)
        r = t["v"].float() * t["vs"].repeat_interleave(256)
        m = f(HYPER["b1"]) * m + f(1 - HYPER["b1"]) * d
        v = f(HYPER["b2"]) * (r * r) + f(1 - HYPER["b2"]) * (d * d)
        # (a root in 64 bits, rounded, is the root rounded; the host's own in 32 bits is not)
        for q, s, x, root in (("m", "ms", m, False), ("v", "vs", torch.sqrt(v.double()).float(), True)):
            b = x.reshape(-1, 256)
            want = b.abs().amax(1) * f(1 / 448)
            assert torch.equal(o[s], want)
            y = b / want[:, None]
            if root:
                y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
            codes = y.reshape(-1).to(FP8).view(torch.uint8)
            assert torch.equal(o[q].view(torch.uint8), codes), (q, int((o[q].view(torch.uint8) != codes).sum()))
            t[q], t[s] = o[q], o[s]
        t["p"] = o["p"]
