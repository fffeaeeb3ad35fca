"""The operators around the layer run together, as a block of a model uses
them: pre-norm, the layer's router, sort, MXFP4 rows, the experts' products,
combine, post-norm with the next block's pre-norm; and the way back.  Also
their calls replayed from a captured HIP graph, on two streams at once, and at
offsets past 32 bits.

Each stage is checked against 64-bit arithmetic on the values that the stage
before left on the GPU (a rounding to four bits turns a last-bit difference
into a whole step), with the bounds of the stages' own tests."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from bit_quantized_routed_router_amd import synthetic as S
from tests.gpu_helpers import SeededLayer
from tests.ops_ref import close, gen, mx_quantize, mx_pack, mx_random, mx_values, rand, sort_slots

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF, F32 = D.DT_BF16, D.DT_F32


class Block:
    """One block: a tiny layer's router, MXFP4 experts, norms with a gate per token."""

    def __init__(self, T, layer, seed=0):
        c = layer.cfg
        self.T, self.d, self.E, self.k, self.f, self.layer = T, c.d, c.E, c.k, c.f, layer
        g = gen(seed)
        self.w = {n: 1 + rand(g, c.d, scale=0.1) for n in ("pre", "post", "next")}
        self.norm = D.Norm(c.d, EPS, 0.5, D.GATE_TOKEN, *(self.w[n].cuda() for n in ("pre", "post", "next")))
        self.mats = {n: [mx_random(g, *s, scale=0.1) for _ in range(c.E)]
                     for n, s in (("gate", (c.f, c.d)), ("up", (c.f, c.d)), ("down", (c.d, c.f)))}
        self.packed = {n: torch.cat([m[0] for m in v]).cuda() for n, v in self.mats.items()}
        self.h, self.gate, self.base = rand(g, T, c.d).cuda(), rand(g, T).cuda(), rand(g, T, c.d).cuda()
        self.dh_out, self.dx_next = rand(g, T, c.d).cuda(), rand(g, T, c.d).cuda()
        self.g = g
        S_, z = T * c.k, lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        i32 = torch.int32
        self.o = dict(x=z(T, c.d, t=torch.bfloat16), idx=z(T, c.k, t=i32), tw=z(T, c.k), counts=z(c.E, t=i32),
                      offsets=z(c.E + 1, t=i32), perm=z(S_, t=i32), inv=z(T, c.k, t=i32),
                      a=z(S_ * c.d * 17 // 32, t=torch.uint8), hid=z(S_, c.f, t=torch.bfloat16),
                      hq=z(S_ * c.f * 17 // 32, t=torch.uint8), ys=z(S_, c.d), y=z(T, c.d), h_out=z(T, c.d),
                      x_next=z(T, c.d, t=torch.bfloat16))
        self.ws_route = layer.layer.workspace(T, D.MODE_ROUTE)
        n = D.group_workspace_bytes(T, c.k, c.E)
        self.ws_group = (z(n, t=torch.uint8), n)
        self.ws_norm = self.norm.workspace(T)
        self.b = dict(dy=z(T, c.d), dgate=z(T), dw_post=z(c.d), dys=z(S_, c.d), dw=z(T, c.k), dl=z(T, c.k),
                      dhid=z(S_, c.f), dx=z(T, c.d), dh=z(T, c.d), dw_pre=z(c.d))

    def forward(self):
        o, T, d, k, E, f, n = self.o, self.T, self.d, self.k, self.E, self.f, self.T * self.k
        D.norm_pre(self.norm.desc, self.h, F32, T, o["x"], BF)
        D.route(self.layer.layer.desc, o["x"], BF, T, o["idx"], o["tw"], None, None, None, *self.ws_route)
        D.group(o["idx"], T, k, E, o["counts"], o["offsets"], o["perm"], o["inv"], *self.ws_group)
        D.mx_quantize(o["x"], BF, T, o["inv"], k, n, d, o["a"])
        D.mx_product(o["a"], n, d, self.packed["gate"], self.packed["up"], f, E, o["offsets"], o["hid"], BF)
        D.mx_quantize(o["hid"], BF, n, None, 1, n, f, o["hq"])
        D.mx_product(o["hq"], n, f, self.packed["down"], None, d, E, o["offsets"], o["ys"], F32)
        D.combine(o["ys"], F32, n, o["inv"], o["tw"], self.base, T, k, d, o["y"], F32)
        D.norm_post(self.norm.desc, self.h, F32, o["y"], F32, self.gate, T, o["h_out"], o["x_next"], BF)

    def backward(self):
        """From the gradient of h_out to those of y, the gate, the routing
        logits, the experts' hidden rows and (through the gate matrix, as a
        linear expert) the block's input."""
        o, b, T, d, k, E, f, n = self.o, self.b, self.T, self.d, self.k, self.E, self.f, self.T * self.k
        D.norm_post_grad(self.norm.desc, self.dh_out, F32, o["y"], F32, self.gate, T, b["dy"], b["dw_post"], b["dgate"],
                         *self.ws_norm)
        D.combine_grad(b["dy"], F32, o["ys"], F32, n, o["inv"], o["tw"], T, k, d, b["dys"], b["dw"], b["dl"])
        D.mx_product_grad(b["dys"], F32, n, d, self.packed["down"], f, E, o["offsets"], b["dhid"], F32)
        # the rows' gradient reuses dys, which the step before has read
        D.mx_product_grad(b["dhid"], F32, n, f, self.packed["gate"], d, E, o["offsets"], b["dys"], F32)
        D.combine(b["dys"], F32, n, o["inv"], None, None, T, k, d, b["dx"], F32)
        D.norm_pre_grad(self.norm.desc, self.h, F32, b["dx"], F32, self.dh_out, T, b["dh"], b["dw_pre"], *self.ws_norm)

    def outputs(self):
        return {**{k: v.clone() for k, v in self.o.items()}, **{k: v.clone() for k, v in self.b.items()}}


@pytest.fixture(scope="module")
def layer():
    return SeededLayer(S.CONFIGS["tiny"], device_quantize=False)


def unpack(p, n, cols):
    p = p.cpu()
    half = n * cols // 2
    code = torch.stack([p[:half] & 15, p[:half] >> 4], 1).reshape(n, cols).long()
    return mx_values(code, p[half:].reshape(n, cols // 32).long())


@pytest.mark.parametrize("T", [1, 7, 40, 150])
def test_block_forward_and_back(layer, T):
    B = Block(T, layer, seed=T)
    B.forward()
    B.backward()
    torch.cuda.synchronize()
    o, b = {n: v.cpu() for n, v in B.o.items()}, {n: v.cpu() for n, v in B.b.items()}
    d, E, k, f, n = B.d, B.E, B.k, B.f, T * B.k
    h = B.h.cpu().double()
    root = (h.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    x = h / root * B.w["pre"].double()
    close(o["x"], x, x.abs(), 100, "x")
    for name, ref in zip(("counts", "offsets", "perm", "inv"), sort_slots(o["idx"], E)):
        assert torch.equal(o[name], ref), name
    # rows in the experts' order, exactly as the format has them
    order = o["perm"].long()
    assert torch.equal(o["a"], mx_pack(*mx_quantize(o["x"][order // k])))
    off = o["offsets"].tolist()
    a = unpack(o["a"], n, d)
    hid, mh = torch.zeros(n, f, dtype=torch.float64), torch.zeros(n, f, dtype=torch.float64)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        G, U_ = B.mats["gate"][e][1], B.mats["up"][e][1]
        gg, uu = a[s] @ G.t(), a[s] @ U_.t()
        hid[s] = gg * torch.sigmoid(gg) * uu
        mh[s] = 2 * d * (1.1 * (a[s].abs() @ G.abs().t()) * uu.abs() + (gg * torch.sigmoid(gg)).abs() *
                         (a[s].abs() @ U_.abs().t())) + (16 + gg.abs()) * hid[s].abs()
    close(o["hid"], hid, mh, 1, "hidden rows")
    assert torch.equal(o["hq"], mx_pack(*mx_quantize(o["hid"])))
    hq = unpack(o["hq"], n, f)
    ys, my = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        ys[s], my[s] = hq[s] @ B.mats["down"][e][1].t(), hq[s].abs() @ B.mats["down"][e][1].abs().t()
    close(o["ys"], ys, my, 2 * f, "ys")
    tw, pos = o["tw"].double(), o["inv"].long()
    terms = tw[:, :, None] * o["ys"].double()[pos]
    base = B.base.cpu().double()
    close(o["y"], base + terms.sum(1), base.abs() + terms.abs().sum(1), 2 * k + 1, "y")
    y, gate = o["y"].double(), B.gate.cpu().double()[:, None]
    q = 1 / (y.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    t = gate * (y * q * B.w["post"].double())
    close(o["h_out"], 0.5 * h + t, (0.5 * h).abs() + t.abs(), 100, "h_out")

    # the way back
    dh_out = B.dh_out.cpu().double()
    u = dh_out * gate * B.w["post"].double()
    dy = q * (u - y * q * q * (y * u).mean(1, keepdim=True))
    close(b["dy"], dy, q * (u.abs() + y.abs() * q * q * (y * u).abs().mean(1, keepdim=True)), 200, "dy")
    dys = tw[:, :, None] * b["dy"].double()[:, None, :]
    dot = (b["dy"].double()[:, None, :] * o["ys"].double()[pos])
    rdw, mdw = dot.sum(2), dot.abs().sum(2)
    close(b["dw"], rdw, mdw, 100, "dw")
    close(b["dl"], tw * (rdw - (tw * rdw).sum(1, keepdim=True)), tw * (mdw + (tw * mdw).sum(1, keepdim=True)), 200, "dl")
    flat = torch.zeros(n, d, dtype=torch.float64)
    flat[pos.reshape(-1)] = dys.reshape(n, d)
    dhid, mhid = torch.zeros(n, f, dtype=torch.float64), torch.zeros(n, f, dtype=torch.float64)
    dxs, mxs = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        W = B.mats["down"][e][1]
        dhid[s], mhid[s] = flat[s] @ W, flat[s].abs() @ W.abs()
        V = B.mats["gate"][e][1]
        dxs[s], mxs[s] = b["dhid"].double()[s] @ V, b["dhid"].double()[s].abs() @ V.abs()
    close(b["dhid"], dhid, mhid, 6 * d + 1, "dhid")  # three parts a term, and dys's own rounding
    close(b["dys"], dxs, mxs, 6 * f, "dxs")
    back = b["dys"].double()[pos]
    close(b["dx"], back.sum(1), back.abs().sum(1), k, "dx")
    r, dx = 1 / root, b["dx"].double()
    v = dx * B.w["pre"].double()
    dh = 0.5 * dh_out + r * (v - h * r * r * (h * v).mean(1, keepdim=True))
    close(b["dh"], dh, 0.5 * dh_out.abs() + r * (v.abs() + h.abs() * r * r * (h * v).abs().mean(1, keepdim=True)), 200, "dh")


def test_graph_replays_match_eager(layer):
    """Two blocks of different sizes, forward and back, captured once and
    replayed three times with other inputs in between; every replay gives the
    eager results bit for bit."""
    blocks = [Block(5, layer, seed=1), Block(90, layer, seed=2)]
    inputs = [[(torch.randn_like(b.h), torch.randn_like(b.dh_out)) for b in blocks] for _ in range(3)]

    def run():
        for b in blocks:
            b.forward()
            b.backward()

    def load(i):
        for b, (h, dh) in zip(blocks, inputs[i]):
            b.h.copy_(h)
            b.dh_out.copy_(dh)

    ref = []
    for i in range(3):
        load(i)
        run()
        torch.cuda.synchronize()
        ref.append([b.outputs() for b in blocks])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in (2, 0, 1):
        load(i)
        for b in blocks:
            for v in (*b.o.values(), *b.b.values()):
                v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for b, want in zip(blocks, ref[i]):
            for name, got in b.outputs().items():
                assert torch.equal(got, want[name]), f"replay with inputs {i}: {name}"
        load((i + 1) % 3)  # eager work of the program's own between replays
        run()
        torch.cuda.synchronize()


def test_two_streams_at_once(layer):
    """Two blocks on two streams without any order between them."""
    blocks = [Block(64, layer, seed=3), Block(33, layer, seed=4)]
    ref = []
    for b in blocks:
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        ref.append(b.outputs())
        for v in (*b.o.values(), *b.b.values()):
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        for s, b in zip(streams, blocks):
            with torch.cuda.stream(s):
                b.forward()
                b.backward()
    torch.cuda.synchronize()
    for b, want in zip(blocks, ref):
        for name, got in b.outputs().items():
            assert torch.equal(got, want[name]), name


def test_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^32 and 2^31: the last rows of
    long tensors against the same rows alone."""
    T, d, k = 600_000, 4096, 1
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    # bit patterns of both signs, their exponent's top bit cleared: finite, below 2
    x.view(torch.int16).random_(-32768, 32767).bitwise_and_(~0x4000)
    tail = x[-70:].clone()
    norm = D.Norm(d, EPS)
    out, few = torch.empty_like(x), torch.empty_like(tail)
    D.norm_pre(norm.desc, x, BF, T, out, BF)
    D.norm_pre(norm.desc, tail, BF, 70, few, BF)
    assert torch.equal(out[-70:], few)
    inv = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda").reshape(T, 1)
    D.dispatch(x, BF, T, k, d, inv, out, T)
    assert torch.equal(out[:70], tail.flip(0)) and torch.equal(out[-1], x[0])
    back = torch.empty_like(x)
    D.combine(out, BF, T, inv, None, None, T, k, d, back, BF)
    assert torch.equal(back[-70:], tail) and torch.equal(back[0], x[0])
    packed = torch.empty(T * d * 17 // 32, dtype=torch.uint8, device="cuda")
    D.mx_quantize(x, BF, T, None, 1, T, d, packed)
    few_packed = torch.empty(70 * d * 17 // 32, dtype=torch.uint8, device="cuda")
    D.mx_quantize(tail, BF, 70, None, 1, 70, d, few_packed)
    D.mx_dequantize(packed, T, d, out, BF)
    D.mx_dequantize(few_packed, 70, d, few, BF)
    assert torch.equal(out[-70:], few)
    del out, back, x
    # products of the last rows: 16 outputs, 2^31 code bytes behind them
    n = 1_100_000
    code = torch.randint(0, 256, (n * d // 2,), dtype=torch.uint8, device="cuda")
    scale = torch.full((n * d // 32,), 120, dtype=torch.uint8, device="cuda")
    a = torch.cat([code, scale])
    w = torch.cat([torch.randint(0, 256, (32 * d // 2,), dtype=torch.uint8, device="cuda"),
                   torch.full((d,), 120, dtype=torch.uint8, device="cuda")])
    y = torch.empty(n, 32, device="cuda")
    D.mx_product(a, n, d, w, None, 32, 1, None, y, F32)
    last = torch.cat([code[-70 * d // 2:], scale[-70 * d // 32:]])
    few = torch.empty(70, 32, device="cuda")
    D.mx_product(last, 70, d, w, None, 32, 1, None, few, F32)
    # the two calls add in different orders: 2 d steps of the terms' magnitude,
    # which 6 * 6 * 2^-14 bounds
    assert (y[-70:] - few).abs().max() <= 2 * d * 2.0 ** -24 * d * 36 * 2.0 ** -14
