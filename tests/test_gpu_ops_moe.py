"""GPU parity of the sort by expert, dispatch and combine (ds4moe_group,
ds4moe_dispatch, ds4moe_combine, ds4moe_combine_grad) with plain loops and
64-bit sums.  The sort, dispatch and rows without a slot are exact.  A
combined value takes k products and sums (k + 1 roundings); a weight's
gradient adds at most 64 products per thread, 6 steps in the wave and 4
waves (100 roundings, 100 more through the softmax's mean)."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests.ops_ref import DT, TYPES, close, gen, rand, sort_slots

pytestmark = pytest.mark.gpu


def draw_idx(g, T, k, E, dead=0.2, repeat=False):
    if repeat:
        idx = torch.randint(0, E, (T, k), generator=g)
    else:
        idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].sort(1).values
    out = torch.tensor([-1, E, -(2 ** 31), 2 ** 31 - 1])[torch.randint(0, 4, (T, k), generator=g)]
    return torch.where(torch.rand(T, k, generator=g) < dead, out, idx).to(torch.int32)


def group(idx, E, ws=None):
    T, k = idx.shape
    i = lambda *n: torch.full(n, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    o = (i(E), i(E + 1), i(T * k), i(T, k))
    n = D.group_workspace_bytes(T, k, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if ws is None else ws
    D.group(idx.cuda(), T, k, E, *o, ws, n)
    return o


def check_group(idx, E, label):
    for name, got, ref in zip(("counts", "offsets", "perm", "inv"), group(idx, E), sort_slots(idx, E)):
        assert torch.equal(got.cpu(), ref), f"{label}: {name}"


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 6, 256), (2, 16, 1024), (16, 6, 256), (63, 1, 3), (64, 1, 64), (65, 2, 65),
                                   (341, 12, 40), (512, 8, 1024), (513, 8, 1023), (683, 6, 256), (1024, 4, 1024),
                                   (2048, 6, 256), (5000, 7, 17), (20000, 16, 512)])
@pytest.mark.parametrize("repeat", [False, True])
def test_group(T, k, E, repeat):
    check_group(draw_idx(gen(T * k + E), T, k, E, 0.2, repeat or k > E), E, f"T={T} k={k} E={E}")


def test_group_largest():
    """2^20 tokens of 16 slots and 1024 experts, against a stable library sort."""
    T, k, E = 1 << 20, 16, 1024
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    idx = torch.randint(-40, E + 40, (T, k), dtype=torch.int32, device="cuda", generator=g)
    counts, offsets, perm, inv = group(idx, E)
    flat = idx.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    assert torch.equal(counts.long(), torch.bincount(key, minlength=E + 1)[:E])
    assert torch.equal(offsets[1:].long(), counts.long().cumsum(0)) and int(offsets[0]) == 0
    live = int(offsets[E])
    assert torch.equal(perm[:live].long(), order[:live]) and (perm[live:] == -1).all()
    want = torch.full((T * k,), -1, dtype=torch.int64, device="cuda")
    want[order[:live]] = torch.arange(live, device="cuda")
    assert torch.equal(inv.reshape(-1).long(), want)


@pytest.mark.parametrize("T", [5, 3000])
def test_group_one_expert_and_none(T):
    check_group(torch.full((T, 3), 9, dtype=torch.int32), 16, "one expert")
    check_group(torch.full((T, 3), -1, dtype=torch.int32), 16, "no expert")
    check_group(torch.full((T, 3), 16, dtype=torch.int32), 16, "expert past the last")


def test_group_matches_route():
    """The layer's own routing and the sort of its indices agree."""
    from bit_quantized_routed_router_amd import synthetic as S
    from tests.gpu_helpers import SeededLayer
    L = SeededLayer(S.CONFIGS["tiny"], device_quantize=False)
    for T in (3, 40):
        r = L.route(L.x(T=T, variant=900 + T))
        counts, offsets, perm, _ = group(torch.from_numpy(r["idx"]), L.cfg.E)
        assert torch.equal(counts.cpu(), torch.from_numpy(r["counts"]))
        assert torch.equal(offsets.cpu(), torch.from_numpy(r["offsets"]))
        assert torch.equal(perm.cpu(), torch.from_numpy(r["perm"]))


class Rows:
    def __init__(self, T, k, E, d, x="f32", ys="f32", y="f32", dead=0.2, spare=3, seed=1):
        g = gen(seed + 7 * T + d)
        self.T, self.k, self.E, self.d, self.kinds = T, k, E, d, dict(x=x, ys=ys, y=y)
        self.idx = draw_idx(g, T, k, E, dead)
        self.inv = sort_slots(self.idx, E)[3]
        self.live = self.inv >= 0
        self.n = T * k + spare
        self.x, self.base = rand(g, T, d, kind=x), rand(g, T, d, kind=y)
        self.ys, self.dy = rand(g, self.n, d, kind=ys), rand(g, T, d, kind=y)
        n_live = int(self.live.sum())
        self.ys[n_live:] = float("nan")  # rows behind the last slot
        w = torch.softmax(torch.where(self.live, rand(g, T, k), torch.tensor(-1e30)), 1)
        self.w = torch.where(self.live, w, torch.tensor(float("nan")))  # never read
        self.dev = {n: getattr(self, n).cuda() for n in ("inv", "x", "base", "ys", "dy", "w")}

    def dispatch(self):
        xs = torch.full((self.n, self.d), 55.0, dtype=TYPES[self.kinds["x"]], device="cuda")
        D.dispatch(self.dev["x"], DT[self.kinds["x"]], self.T, self.k, self.d, self.dev["inv"], xs, self.n)
        return xs

    def combine(self, w=True, base=True, y=None):
        y = torch.full((self.T, self.d), float("nan"), dtype=TYPES[self.kinds["y"]], device="cuda") if y is None else y
        b = self.dev["base"] if base is True else base
        D.combine(self.dev["ys"], DT[self.kinds["ys"]], self.n, self.dev["inv"], self.dev["w"] if w else None,
                  b or None if b is False else b, self.T, self.k, self.d, y, DT[self.kinds["y"]])
        return y

    def grad(self, w=True, want=(True, True, True), dys=None):
        new = [torch.full((self.n, self.d), 55.0, dtype=TYPES[self.kinds["ys"]], device="cuda") if dys is None else dys,
               torch.full((self.T, self.k), float("nan"), device="cuda"),
               torch.full((self.T, self.k), float("nan"), device="cuda")]
        o = [t if on else None for t, on in zip(new, want)]
        ys = self.dev["ys"] if dys is None else dys
        D.combine_grad(self.dev["dy"], DT[self.kinds["y"]], ys, DT[self.kinds["ys"]], self.n, self.dev["inv"],
                       self.dev["w"] if w else None, self.T, self.k, self.d, *o)
        return o

    # ---- references
    def slots(self):
        """(token, slot in it, position) of the slots with a row"""
        t, j = self.live.nonzero(as_tuple=True)
        return t, j, self.inv[t, j].long()

    def w64(self, w):
        return torch.where(self.live, self.w if w else torch.ones(()), torch.zeros(())).double()

    def check(self):
        label = f"T={self.T} k={self.k} E={self.E} d={self.d} {self.kinds}"
        t, j, p = self.slots()
        want = torch.full((self.n, self.d), 55.0, dtype=self.x.dtype)
        want[p] = self.x[t]
        assert torch.equal(self.dispatch().cpu(), want), label + ": dispatch"
        rows = torch.zeros(self.T, self.k, self.d, dtype=torch.float64)
        rows[t, j] = self.ys[p].double()
        for w in (True, False):
            w64 = self.w64(w)
            for base in (True, False):
                b = self.base.double() if base else torch.zeros(self.T, self.d, dtype=torch.float64)
                terms = w64[:, :, None] * rows
                close(self.combine(w, base), b + terms.sum(1), b.abs() + terms.abs().sum(1), 2 * self.k + 1,
                      f"{label} combine w={w} base={base}")
            dys, dw, dl = self.grad(w)
            dy = self.dy.double()
            ref = torch.full((self.n, self.d), 55.0, dtype=torch.float64)
            ref[p] = (w64[:, :, None] * dy[:, None, :])[t, j]
            close(dys, ref, ref.abs(), 1, label + " dys")
            prod = rows * dy[:, None, :]
            rdw, mdw = prod.sum(2), prod.abs().sum(2)
            close(dw, rdw, mdw, 100, label + " dw")
            mean = (w64 * rdw).sum(1, keepdim=True)
            mm = (w64 * mdw).sum(1, keepdim=True)
            close(dl, w64 * (rdw - mean), w64 * (mdw + mm), 200, label + " dlogits")
            dead = ~self.live
            assert (dw.cpu()[dead] == 0).all() and (dl.cpu()[dead] == 0).all()


@pytest.mark.parametrize("x,ys,y", [("f32", "f32", "f32"), ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"),
                                    ("f32", "bf16", "bf16")])
def test_rows_types(x, ys, y):
    Rows(13, 6, 24, 768, x, ys, y).check()


@pytest.mark.parametrize("T,k,E,d,dead", [(1, 1, 1, 256, 0.0), (1, 6, 256, 4096, 0.0), (1, 3, 8, 256, 1.0), (3, 16, 64, 2304, 0.3),
                                          (129, 5, 7, 512, 0.5), (4, 2, 4, 16384, 0.1), (9, 4, 9, 8448, 0.2),
                                          (300, 1, 40, 256, 0.9)])
def test_rows_sizes(T, k, E, d, dead):
    Rows(T, k, E, d, "bf16", "f32", "f32", dead).check()


def test_combine_in_place_and_partial_outputs():
    r = Rows(21, 4, 12, 512, "f32", "bf16", "f32")
    ref = r.combine()
    y = r.dev["base"].clone()
    assert torch.equal(r.combine(base=y, y=y), ref)
    dys, dw, dl = r.grad()
    for want in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        for a, b in zip(r.grad(want=want), (dys, dw, dl)):
            assert a is None or torch.equal(a, b)
    buf = r.dev["ys"].clone()
    got = r.grad(dys=buf)
    n = int(r.live.sum())
    assert torch.equal(got[0][:n], dys[:n]) and torch.equal(got[1], dw) and got[0][n:].isnan().all()


def test_positions_out_of_range_are_skipped():
    """Positions past the rows that the call names are taken as none."""
    r = Rows(8, 2, 4, 256, dead=0.0)
    r.inv[2, 1], r.inv[5, 0], r.inv[6, 1] = r.n, 2 ** 31 - 1, -7
    r.live = (r.inv >= 0) & (r.inv < r.n)
    r.dev["inv"] = r.inv.cuda()
    r.check()


def test_dispatch_and_combine_are_each_others_gradient():
    """<dispatch(x), g> = <x, combine(g)> with weights of one, the 64-bit sums of
    both sides from the kernels' fp32 rows, to the roundings of k sums."""
    r = Rows(50, 3, 10, 512)
    n = int(r.live.sum())
    xs, g = r.dispatch()[:n].double(), r.dev["ys"][:n].double()
    back = r.combine(w=False, base=False).double()
    prod = r.dev["x"].double() * back
    a, b = float((xs * g).sum()), float(prod.sum())
    assert abs(a - b) <= 8 * 2.0 ** -24 * float((xs.abs() * g.abs()).sum())


def test_dlogits_against_differences():
    """dlogits against central differences of the 64-bit loss <y, dy> through the
    softmax (step 1e-4: remainder below 1e-6 of the terms)."""
    r = Rows(6, 4, 8, 256, dead=0.3)
    _, _, dl = r.grad()
    t, j, p = r.slots()
    rows = torch.zeros(r.T, r.k, r.d, dtype=torch.float64)
    rows[t, j] = r.ys[p].double()
    dot = (rows * r.dy.double()[:, None, :]).sum(2)
    logit = torch.where(r.live, torch.where(r.live, r.w, torch.ones(())).double().log(), torch.tensor(-1e30).double())

    def loss(l):
        return float((torch.softmax(l, 1) * dot).sum())

    v = torch.where(r.live, torch.randn(r.T, r.k, generator=gen(3), dtype=torch.float64), torch.zeros(()).double())
    want = (loss(logit + 1e-4 * v) - loss(logit - 1e-4 * v)) / 2e-4
    prod = dl.cpu().double() * v
    assert abs(float(prod.sum()) - want) <= 2e-6 * float((dot.abs() * v.abs()).sum())
