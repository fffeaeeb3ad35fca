"""GPU parity of the MXFP4 rows and products (ds4moe_mx_*) with the format's
definition and 64-bit sums.  Codes, scales and values read back are exact.  A
product's terms are exact (two FP4 values, powers of two) and its sum is fp32
in whatever order and rounding: one step (2 half steps) per term at most.
silu(g) u: the exponential's argument is off by |g| half steps and the rest
by less than 16, and the two sums enter with |silu'| <= 1.1.  The fp32 form
of the gradient adds three exact parts per value: 3 terms each."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests.ops_ref import (DT, TYPES, U, close, gen, mx_pack, mx_quantize, mx_random, mx_values, rand, random_offsets,
                           sort_slots)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rows
def awkward_rows(kind):
    """Rows of ties, signs, zeros, subnormals, the type's largest and smallest
    values, mixed magnitudes, infinities and NaN."""
    g = gen(5)
    t = TYPES[kind]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    near = torch.cat([ties, ties * (1 - 2.0 ** -7), ties * (1 + 2.0 ** -7), -ties])
    rows = [torch.cat([near * 2.0 ** e for e in range(-4, 4)]),
            torch.cat([torch.full((32,), 4.0) * torch.linspace(-1, 1, 32) * 2.0 ** e for e in (-126, -120, 0, 90, 100, 110, 120, 125)]),
            torch.zeros(256), -torch.zeros(256),
            rand(g, 256) * torch.exp2(torch.randint(-140, 120, (256,), generator=g).float()),
            rand(g, 256) * 2.0 ** -130,
            torch.exp2(torch.arange(256).float() - 149).clamp(max=torch.finfo(t).max),
            torch.full((256,), torch.finfo(t).max), torch.full((256,), -torch.finfo(t).max),
            torch.full((256,), torch.finfo(t).tiny)]
    x = torch.stack(rows).to(t)
    bad = rand(g, 3, 256).to(t)
    bad[0, 40] = float("nan")
    bad[1, 64] = float("inf")
    bad[2, 255] = -float("inf")
    return torch.cat([x, bad])


def quantize(x, inv=None, n=None, k=1):
    T, cols = x.shape
    n = T if n is None else n
    out = torch.full((n * cols * 17 // 32,), 0xA5, dtype=torch.uint8, device="cuda")
    kind = "bf16" if x.dtype == torch.bfloat16 else "f32"
    D.mx_quantize(x.cuda(), DT[kind], T, None if inv is None else inv.cuda(), k, n, cols, out)
    return out


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_awkward_values(kind):
    x = awkward_rows(kind)
    code, sc = mx_quantize(x)
    got = quantize(x)
    want = mx_pack(code, sc)
    half = x.numel() // 2
    assert torch.equal(got.cpu()[half:], want[half:]), "scales"
    assert torch.equal(got.cpu()[:half], want[:half]), "codes"
    for out in ("f32", "bf16"):
        v = torch.empty(x.shape, dtype=TYPES[out], device="cuda")
        D.mx_dequantize(got, x.shape[0], x.shape[1], v, DT[out])
        ref = mx_values(code, sc).to(TYPES[out])
        same = (v.cpu() == ref) | (v.cpu().isnan() & ref.isnan())
        assert same.all(), out


@pytest.mark.parametrize("T,cols", [(1, 256), (3, 768), (1, 4096), (130, 2304), (2, 16384)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_equals_the_codec(T, cols, kind):
    x = (rand(gen(T + cols), T, cols) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=gen(1)).float())).to(TYPES[kind])
    got = quantize(x)
    ref = torch.empty_like(got)
    D.quantize(D.FMT_MXFP4, x.float().cuda(), T, cols, ref)
    assert torch.equal(got, ref)
    v, vr = (torch.empty(T, cols, device="cuda") for _ in range(2))
    D.mx_dequantize(got, T, cols, v, D.DT_F32)
    D.dequantize(D.FMT_MXFP4, got, T, cols, vr)
    assert torch.equal(v, vr)


def test_dequantize_every_code_and_scale():
    """All 16 codes under all 256 scale codes."""
    code = torch.arange(16).repeat(256, 16)
    sc = torch.arange(256)[:, None].repeat(1, 8)
    p = mx_pack(code, sc).cuda()
    for kind in ("f32", "bf16"):
        v = torch.empty(256, 256, dtype=TYPES[kind], device="cuda")
        D.mx_dequantize(p, 256, 256, v, DT[kind])
        ref = mx_values(code, sc).to(TYPES[kind])
        assert ((v.cpu() == ref) | (v.cpu().isnan() & ref.isnan())).all(), kind


def test_quantize_at_sorted_rows():
    """Rows land where the sort says; slots without a row and positions out of
    range write nothing; rows without a slot are left as they were."""
    T, k, E, cols = 37, 3, 8, 512
    g = gen(8)
    idx = torch.where(torch.rand(T, k, generator=g) < 0.3, -1, torch.randint(0, E, (T, k), generator=g)).to(torch.int32)
    inv = sort_slots(idx, E)[3]
    n = T * k
    inv[4, 1], inv[7, 2] = n, 2 ** 31 - 1
    x = rand(g, T, cols, kind="bf16")
    got = quantize(x, inv, n, k).cpu()
    code, sc = mx_quantize(x)
    want_c = torch.full((n, cols // 2), 0xA5, dtype=torch.uint8)
    want_s = torch.full((n, cols // 32), 0xA5, dtype=torch.uint8)
    c2 = code.reshape(T, cols // 2, 2)
    packed = (c2[..., 0] | (c2[..., 1] << 4)).to(torch.uint8)
    for t in range(T):
        for j in range(k):
            p = int(inv[t, j])
            if 0 <= p < n:
                want_c[p], want_s[p] = packed[t], sc[t].to(torch.uint8)
    assert torch.equal(got, torch.cat([want_c.reshape(-1), want_s.reshape(-1)]))


# ---------------------------------------------------------------- products
class Product:
    def __init__(self, n, rows, cols, E=1, tail=0, glu=False, offsets=None, seed=2, scale=0.3):
        g = gen(seed + n + rows + cols + E)
        self.n, self.rows, self.cols, self.E, self.glu = n, rows, cols, E, glu
        self.a, self.a64 = mx_random(g, n, cols)
        self.w, self.w64 = [], []
        for _ in range(2 if glu else 1):
            mats = [mx_random(g, rows, cols, scale) for _ in range(E)]
            self.w.append(torch.cat([m[0] for m in mats]))
            self.w64.append([m[1] for m in mats])
        self.offsets = random_offsets(g, n, E, tail) if offsets is None else torch.tensor(offsets, dtype=torch.int32)
        self.g = g

    def run(self, kind="f32", offsets=True, stream=None):
        y = torch.full((self.n, self.rows), 55.0, dtype=TYPES[kind], device="cuda")
        w = [t.cuda() for t in self.w]
        off = self.offsets.cuda() if offsets else None
        D.mx_product(self.a.cuda(), self.n, self.cols, w[0], w[1] if self.glu else None, self.rows, self.E, off, y, DT[kind])
        torch.cuda.synchronize()
        return y

    def ref(self):
        y = torch.full((self.n, self.rows), 55.0, dtype=torch.float64)
        m = torch.zeros_like(y)
        off = self.offsets.clamp(0, self.n).tolist()
        for e in range(self.E):
            lo, hi = off[e], off[e + 1]
            if hi <= lo:
                continue
            a = self.a64[lo:hi]
            p = [a @ w[e].t() for w in self.w64]
            q = [a.abs() @ w[e].abs().t() for w in self.w64]
            if self.glu:
                s = p[0] * torch.sigmoid(p[0])
                y[lo:hi] = s * p[1]
                # magnitudes in units of half steps
                m[lo:hi] = 2 * self.cols * (1.1 * q[0] * p[1].abs() + s.abs() * q[1]) + (16 + p[0].abs()) * y[lo:hi].abs()
            else:
                y[lo:hi], m[lo:hi] = p[0], 2 * self.cols * q[0]
        return y, m

    def check(self, kinds=("f32", "bf16"), offsets=True):
        y, m = self.ref()
        for kind in kinds:
            close(self.run(kind, offsets), y, m, 1,
                  f"n={self.n} rows={self.rows} cols={self.cols} E={self.E} glu={self.glu} {kind}")


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n,rows,cols", [(1, 16, 256), (1, 48, 512), (2, 272, 768), (15, 32, 1024), (16, 528, 256), (17, 64, 1280),
                                         (33, 16, 2304), (63, 144, 512), (64, 256, 256), (65, 80, 768), (129, 528, 512),
                                         (130, 256, 1792), (257, 272, 1024), (300, 512, 768)])
def test_product_dense(n, rows, cols, glu):
    Product(n, rows, cols, glu=glu).check(offsets=False)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n,rows,cols,E,tail", [(1, 32, 256, 256, 0), (6, 256, 512, 256, 0), (96, 64, 768, 40, 3), (50, 48, 256, 1024, 0),
                                                (200, 272, 512, 5, 17), (300, 128, 1024, 3, 0), (700, 96, 256, 9, 1),
                                                (20, 16, 256, 4, 20), (1200, 256, 256, 6, 100)])
def test_product_grouped(n, rows, cols, E, tail, glu):
    """Experts with no row, one row and many; rows behind the last expert stay."""
    Product(n, rows, cols, E, tail, glu).check(("f32",) if glu else ("bf16", "f32"))


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n,rows,cols,E,tail", [(70, 1040, 768, 40, 5), (1290, 2064, 256, 5, 7), (2050, 4112, 512, 1, 0),
                                                (777, 1552, 1280, 3, 0), (5000, 4096, 256, 9, 3), (40, 8208, 256, 1, 0)])
def test_product_every_tile_size(n, rows, cols, E, tail, glu):
    """Enough outputs for each of the kernels' tile sizes (16, 64, 128 and 256
    rows), with partly filled tiles of rows and outputs."""
    Product(n, rows // 2 // 16 * 16 if glu else rows, cols, E, tail, glu).check(("bf16",))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n,rows,cols,E", [(3100, 4112, 512, 1), (3100, 4096, 768, 1), (3000, 4096, 256, 3)])
def test_product_largest_tiles(n, rows, cols, E, glu, kind):
    """Enough tiles of 256 rows by 256 weight rows to fill the chip, an odd
    number of column pieces and parts past the last output among them."""
    Product(n, rows // 32 * 16 + 16 * (rows % 32 > 0) if glu else rows, cols, E, 3, glu).check((kind,))


def test_product_bad_offsets_stay_in_range():
    """Offsets below zero, past the rows or descending: held to the rows, runs
    that descend are empty."""
    n = 40
    p = Product(n, 32, 256, 6, offsets=[-5, 3, 3, 30, 20, 99, 2 ** 31 - 1])
    y, m = p.ref()
    got = p.run()
    off = p.offsets.clamp(0, n).tolist()
    hit = torch.zeros(n, dtype=torch.int)
    for e in range(6):
        hit[off[e]:max(off[e], off[e + 1])] += 1
    once = hit == 1  # rows of one run only
    close(got.cpu()[once], y[once], m[once], 1, "rows of one run")
    assert (got.cpu()[hit == 0] == 55).all()


def test_product_scale_codes_and_nan():
    """Scale codes over their whole range on both sides: sums in fp32's range
    are met, a block marked NaN makes its row's outputs NaN and no others."""
    n, rows, cols = 20, 32, 512
    p = Product(n, rows, cols)
    half_a, half_w = n * cols // 2, rows * cols // 2
    sa, sw = p.a[half_a:].reshape(n, -1), p.w[0][half_w:].reshape(rows, -1)
    for i in range(n):
        sa[i] = min(254, 13 * i)
    for r in range(rows):
        sw[r] = max(0, 150 - 7 * r)
    sa[3, 5] = 255
    sw[6, 2] = 255
    code = lambda t, m, h: torch.stack([t[:h] & 15, t[:h] >> 4], 1).reshape(m, cols).long()  # noqa: E731
    p.a64 = mx_values(code(p.a, n, half_a), sa.long())
    p.w64[0][0] = mx_values(code(p.w[0], rows, half_w), sw.long())
    y = p.run().cpu()
    ref, m = p.ref()
    assert y[3].isnan().all() and y[:, 6].isnan().all()
    ok = (m < 2.0 ** 126) & (m > 2.0 ** -100) & ~ref.isnan()
    assert ok.sum() > 100
    close(y[ok], ref[ok], m[ok], 1, "scales")
    # no NaN elsewhere, but for sums whose terms pass fp32's range: partial sums
    # of both signs may each be infinite there, and infinity less infinity is NaN
    rest = m < 2.0 ** 126
    rest[3], rest[:, 6] = False, False
    assert rest.sum() > 300 and not y[rest].isnan().any()


def test_product_rows_behind_the_last_expert_are_not_read():
    p = Product(60, 48, 512, 4, tail=30)
    ref = p.run()
    p.a[60 * 256:].reshape(60, 16)[30:] = 255
    assert torch.equal(p.run(), ref)


class Back:
    def __init__(self, n, rows, cols, E=1, tail=0, kind="bf16", offsets=None, seed=4):
        g = gen(seed + n + rows + cols + E)
        self.n, self.rows, self.cols, self.E, self.kind = n, rows, cols, E, kind
        mats = [mx_random(g, rows, cols, 0.1) for _ in range(E)]
        self.w, self.w64 = torch.cat([m[0] for m in mats]), [m[1] for m in mats]
        self.dy = rand(g, n, rows, kind=kind)
        self.offsets = random_offsets(g, n, E, tail) if offsets is None else torch.tensor(offsets, dtype=torch.int32)

    def run(self, out="f32", offsets=True):
        da = torch.full((self.n, self.cols), 55.0, dtype=TYPES[out], device="cuda")
        D.mx_product_grad(self.dy.cuda(), DT[self.kind], self.n, self.rows, self.w.cuda(), self.cols, self.E,
                          self.offsets.cuda() if offsets else None, da, DT[out])
        torch.cuda.synchronize()
        return da

    def check(self, outs=("f32", "bf16"), offsets=True):
        y = torch.full((self.n, self.cols), 55.0, dtype=torch.float64)
        m = torch.zeros_like(y)
        off = self.offsets.tolist()
        for e in range(self.E):
            lo, hi = off[e], off[e + 1]
            y[lo:hi] = self.dy[lo:hi].double() @ self.w64[e]
            m[lo:hi] = self.dy[lo:hi].double().abs() @ self.w64[e].abs()
        parts = 1 if self.kind == "bf16" else 3
        for out in outs:
            close(self.run(out, offsets), y, m, 2 * parts * self.rows,
                  f"back n={self.n} rows={self.rows} cols={self.cols} E={self.E} {self.kind} {out}")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,cols", [(1, 16, 256), (1, 80, 512), (7, 144, 768), (16, 64, 256), (17, 48, 1024), (33, 528, 256),
                                         (64, 256, 512), (65, 272, 256), (200, 96, 768), (129, 512, 1280)])
def test_product_grad_dense(n, rows, cols, kind):
    Back(n, rows, cols, kind=kind).check(offsets=False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,cols,E,tail", [(1, 32, 256, 256, 0), (6, 256, 512, 64, 0), (96, 64, 256, 40, 3), (300, 128, 512, 3, 0),
                                                (700, 96, 256, 9, 50), (20, 16, 256, 4, 20)])
def test_product_grad_grouped(n, rows, cols, E, tail, kind):
    Back(n, rows, cols, E, tail, kind).check()


def test_product_grad_is_the_products_gradient():
    """<y(a), dy> = <a, da(dy)> for the linear product (both sides in 64 bits from
    the kernels' fp32 outputs)."""
    n, rows, cols, E = 50, 64, 512, 3
    p = Product(n, rows, cols, E)
    b = Back(n, rows, cols, E, kind="f32", offsets=p.offsets.tolist())
    b.w, b.w64 = p.w[0], p.w64[0]
    y, da = p.run().cpu().double(), b.run().cpu().double()
    lhs, rhs = float((y * b.dy.double()).sum()), float((p.a64 * da).sum())
    mag = float((p.ref()[1] * b.dy.double().abs()).sum())  # already counts the steps of each sum
    assert abs(lhs - rhs) <= 4 * U * mag


def test_product_grad_extreme_values():
    """Infinities and NaN of dY stay in their row (times zero they are NaN); the
    largest and smallest fp32 values pass through their three parts."""
    n, rows, cols = 6, 32, 256
    b = Back(n, rows, cols, kind="f32")
    b.dy[0] = 0
    b.dy[0, 0] = 3.0e38
    b.dy[1] = 0
    b.dy[1, 5] = 1.0e-30
    b.dy[2, 3] = float("nan")
    b.dy[3, 3] = float("inf")
    got = b.run(offsets=False).cpu()
    w = b.w64[0]
    for row, i in ((0, 0), (1, 5)):
        ref = b.dy[row, i].double() * w[i]
        ok = ref.abs() < 3e38
        close(got[row][ok], ref[ok], ref[ok].abs(), 6, f"row {row}")
    assert got[2].isnan().all()
    assert not torch.isfinite(got[3]).any()
    assert torch.isfinite(got[[1, 4, 5]]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_product_grad_scale_codes(kind):
    """Scale codes from 0 (weights down to 2^-128, bfloat16's subnormal numbers)
    to 220, with dY of a size that brings every product near one (2^120 at
    most, and down to 2^-95, where an fp32 value's three parts are all normal);
    a block marked NaN makes its 32 columns NaN and no others."""
    n, rows, cols = 24, 224, 512
    b = Back(n, rows, cols, kind=kind)
    half = rows * cols // 2
    sc = torch.arange(rows).clamp(max=220)[:, None].repeat(1, cols // 32)
    b.w[half:] = sc.reshape(-1).to(torch.uint8)
    code = torch.stack([b.w[:half] & 15, b.w[:half] >> 4], 1).reshape(rows, cols).long()
    b.w64[0] = mx_values(code, sc)
    b.dy = (b.dy.float().clamp(-3, 3) * torch.exp2((127 - sc[:, 0]).clamp(max=118).float())).to(b.dy.dtype)
    b.check(offsets=False)
    b.w.view(torch.uint8)[half + 5 * (cols // 32) + 3] = 255
    got = b.run(offsets=False).cpu()
    assert got[:, 96:128].isnan().all()
    assert torch.isfinite(got[:, :96]).all() and torch.isfinite(got[:, 128:]).all()


def test_product_grad_bad_offsets_stay_in_range():
    n = 40
    b = Back(n, 48, 256, 6, offsets=[-5, 3, 3, 30, 20, 99, 2 ** 31 - 1])
    got = b.run().cpu()
    off = b.offsets.clamp(0, n).tolist()
    hit = torch.zeros(n, dtype=torch.int)
    owner = torch.zeros(n, dtype=torch.int)
    for e in range(6):
        hit[off[e]:max(off[e], off[e + 1])] += 1
        owner[off[e]:max(off[e], off[e + 1])] = e
    for p in range(n):
        if hit[p] == 0:
            assert (got[p] == 55).all()
        elif hit[p] == 1:
            W = b.w64[int(owner[p])]
            close(got[p], b.dy[p].double() @ W, b.dy[p].double().abs() @ W.abs(), 2 * 48, f"row {p}")


@pytest.mark.parametrize("n,rows,cols,E", [(300, 48, 256, 1), (4100, 32, 4096, 40), (2600, 64, 1024, 20)])
def test_product_grad_every_tile_size(n, rows, cols, E):
    """Tiles of 32 and of 64 rows, partly filled ones among them."""
    Back(n, rows, cols, E, 5).check(("bf16",))


@pytest.mark.parametrize("n,E", [(3000, 1024), (20000, 1024), (9000, 300)])
def test_product_many_experts(n, E):
    """Up to 1024 experts (four to a thread in the search for a tile), most of
    the rows with one of them."""
    g = gen(n)
    cut = torch.randint(0, n, (E - 1,), generator=g).sort().values
    cut[E // 2:] = torch.maximum(cut[E // 2:], torch.tensor(n - E))
    cut[:E // 2] = cut[:E // 2].clamp(max=E)
    off = [0] + cut.sort().values.tolist() + [n]
    p = Product(n, 16, 256, E, offsets=off)
    p.check(("f32",))
    b = Back(n, 16, 256, E, offsets=off)
    b.check(("f32",))


@pytest.mark.parametrize("n", [5, 90, 1500])
def test_largest_matrix(n):
    """16384 x 16384 weights: the first and last outputs, and the gradient's
    first and last columns, of every tile size's forms."""
    m = 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    draw = lambda k: torch.randint(0, 256, (k,), dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    scale = lambda k: torch.randint(112, 124, (k,), dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    w = torch.cat([draw(m * m // 2), scale(m * m // 32)])
    a = torch.cat([draw(n * m // 2), scale(n * m // 32)])
    w16, a16 = (torch.empty(k, m, dtype=torch.bfloat16, device="cuda") for k in (m, n))
    D.mx_dequantize(w, m, m, w16, D.DT_BF16)
    D.mx_dequantize(a, n, m, a16, D.DT_BF16)
    pick = torch.cat([torch.arange(40), torch.arange(m - 40, m)]).cuda()
    y = torch.empty(n, m, device="cuda")
    D.mx_product(a, n, m, w, None, m, 1, None, y, D.DT_F32)
    ws, a64 = w16[pick].double(), a16.double()
    close(y[:, pick], a64 @ ws.t().contiguous(), a64.abs() @ ws.abs().t().contiguous(), 2 * m, "product")
    da = torch.empty(n, m, device="cuda")
    D.mx_product_grad(a16, D.DT_BF16, n, m, w, m, 1, None, da, D.DT_F32)
    wc = w16[:, pick].double()
    close(da[:, pick], a64 @ wc, a64.abs() @ wc.abs(), 2 * m, "gradient")
