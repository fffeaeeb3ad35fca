"""Host-side checks of the operators around the layer (no device work):
sizes of workspaces, and calls that are refused before anything is launched."""
import ctypes

import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D

A = 0x10000  # stand-in device address: aligned, never dereferenced
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def desc(**kw):
    v = dict(d_model=4096, eps=1e-6, res_scale=1.0, gate=D.GATE_NONE, w_pre=A, w_post=A, w_next=A)
    v.update(kw)
    return D.NormDesc(*(v[f[0]] for f in D.NormDesc._fields_))


def status(name, *args):
    return getattr(D.lib(), "ds4moe_" + name)(*args)


BAD_DESC = [(dict(eps=0.0), D.EINVAL), (dict(eps=-1.0), D.EINVAL), (dict(eps=NAN), D.EINVAL), (dict(eps=INF), D.EINVAL),
            (dict(res_scale=NAN), D.EINVAL), (dict(gate=4), D.EINVAL), (dict(gate=-1), D.EINVAL),
            (dict(d_model=300), D.ESHAPE), (dict(d_model=0), D.ESHAPE), (dict(d_model=16640), D.ESHAPE),
            (dict(w_pre=A + 4), D.EALIGN), (dict(w_post=A + 8), D.EALIGN), (dict(w_next=A + 2), D.EALIGN)]


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_norm_descriptor_errors(kw, code):
    n = ctypes.byref(desc(**kw))
    gate = A if kw.get("gate") else None
    assert status("norm_pre", n, A, 0, 1, A, 1, None) == code
    assert status("norm_post", n, A, 0, A, 0, gate, 1, A, A, 1, None) == code
    assert status("norm_pre_grad", n, A, 0, A, 0, A, 1, A, A, A, BIG, None) == code
    assert status("norm_post_grad", n, A, 0, A, 0, gate, 1, A, A, None, A, BIG, None) == code
    assert D.norm_workspace_bytes(desc(**kw), 1) == 0


def test_norm_argument_errors():
    def pre(h=A, hd=0, T=1, x=A, xd=1, n=desc()):
        return status("norm_pre", ctypes.byref(n) if n else None, h, hd, T, x, xd, None)

    def post(h=A, hd=0, y=A, yd=0, gate=None, T=1, ho=A, x=A, xd=1, n=desc()):
        return status("norm_post", ctypes.byref(n), h, hd, y, yd, gate, T, ho, x, xd, None)

    def pre_grad(h=A, dx=A, dho=A, T=1, dh=A, dw=A, ws=A, nb=BIG, hd=0, xd=1, n=desc()):
        return status("norm_pre_grad", ctypes.byref(n), h, hd, dx, xd, dho, T, dh, dw, ws, nb, None)

    def post_grad(dho=A, y=A, gate=None, T=1, dy=A, dw=A, dg=None, ws=A, nb=BIG, hd=0, yd=1, n=desc()):
        return status("norm_post_grad", ctypes.byref(n), dho, hd, y, yd, gate, T, dy, dw, dg, ws, nb, None)

    assert pre(n=None) == D.EINVAL
    for kw in (dict(h=None), dict(x=None), dict(hd=2), dict(xd=-1)):
        assert pre(**kw) == D.EINVAL, kw
    for T in (0, -1, (1 << 20) + 1):
        assert pre(T=T) == D.ESHAPE and post(T=T) == D.ESHAPE
        assert pre_grad(T=T) == D.ESHAPE and post_grad(T=T) == D.ESHAPE
        assert D.norm_workspace_bytes(desc(), T) == 0
    assert pre(h=A + 8) == D.EALIGN and pre(x=A + 2) == D.EALIGN
    for kw in (dict(h=None), dict(y=None), dict(ho=None), dict(yd=3), dict(xd=3), dict(gate=A),
               dict(n=desc(gate=D.GATE_TOKEN)), dict(n=desc(gate=D.GATE_FULL))):
        assert post(**kw) == D.EINVAL, kw
    for kw in (dict(h=A + 4), dict(y=A + 4), dict(ho=A + 4), dict(x=A + 4),
               dict(n=desc(gate=D.GATE_CHANNEL), gate=A + 4), dict(n=desc(gate=D.GATE_TOKEN), gate=A + 2)):
        assert post(**kw) == D.EALIGN, kw
    for kw in (dict(h=None), dict(dx=None), dict(dh=None), dict(ws=None), dict(hd=9)):
        assert pre_grad(**kw) == D.EINVAL, kw
    for kw in (dict(h=A + 4), dict(dx=A + 4), dict(dho=A + 4), dict(dh=A + 4), dict(dw=A + 4), dict(ws=A + 16)):
        assert pre_grad(**kw) == D.EALIGN, kw
    need = D.norm_workspace_bytes(desc(), 100)
    assert need > 0 and pre_grad(T=100, nb=need - 1) == D.EWORKSPACE and post_grad(T=100, nb=need - 1) == D.EWORKSPACE
    g = desc(gate=D.GATE_CHANNEL)
    for kw in (dict(dho=None), dict(y=None), dict(dy=None), dict(dg=A), dict(gate=A), dict(n=g), dict(ws=None),
               dict(n=g, gate=A, dw=None, dg=A, ws=None)):
        assert post_grad(**kw) == D.EINVAL, kw
    for kw in (dict(dho=A + 4), dict(y=A + 4), dict(dy=A + 4), dict(dw=A + 4), dict(n=g, gate=A, dg=A + 4)):
        assert post_grad(**kw) == D.EALIGN, kw


def test_group_argument_errors():
    def group(idx=A, T=4, k=2, E=8, c=A, o=A, p=A, i=A, ws=A, nb=BIG):
        return status("group", idx, T, k, E, c, o, p, i, ws, nb, None)

    for kw in (dict(idx=None), dict(c=None), dict(o=None), dict(p=None), dict(i=None), dict(ws=None)):
        assert group(**kw) == D.EINVAL, kw
    for kw in (dict(T=0), dict(T=(1 << 20) + 1), dict(k=0), dict(k=17), dict(E=0), dict(E=1025)):
        assert group(**kw) == D.ESHAPE, kw
        assert D.group_workspace_bytes(kw.get("T", 4), kw.get("k", 2), kw.get("E", 8)) == 0
    for kw in (dict(idx=A + 2), dict(c=A + 1), dict(o=A + 2), dict(p=A + 2), dict(i=A + 2), dict(ws=A + 16)):
        assert group(**kw) == D.EALIGN, kw
    for T in (1, 100000):
        need = D.group_workspace_bytes(T, 6, 256)
        assert need > 0 and need % 256 == 0
        assert group(T=T, k=6, E=256, nb=need - 1) == D.EWORKSPACE


def test_row_argument_errors():
    def dispatch(x=A, dt=0, T=4, k=2, d=256, inv=A, xs=A, n=8):
        return status("dispatch", x, dt, T, k, d, inv, xs, n, None)

    def combine(ys=A, sd=0, n=8, inv=A, w=A, base=A, T=4, k=2, d=256, y=A, yd=0):
        return status("combine", ys, sd, n, inv, w, base, T, k, d, y, yd, None)

    def grad(dy=A, yd=0, ys=A, sd=0, n=8, inv=A, w=A, T=4, k=2, d=256, dys=A, dw=A, dl=A):
        return status("combine_grad", dy, yd, ys, sd, n, inv, w, T, k, d, dys, dw, dl, None)

    for f in (dispatch, combine, grad):
        for kw in (dict(T=0), dict(T=-3), dict(T=(1 << 20) + 1), dict(k=0), dict(k=17), dict(d=128), dict(d=16640),
                   dict(n=0), dict(n=(1 << 24) + 1)):
            assert f(**kw) == D.ESHAPE, (f.__name__, kw)
        assert f(inv=None) == D.EINVAL and f(inv=A + 2) == D.EALIGN
    for kw in (dict(x=None), dict(xs=None), dict(dt=2)):
        assert dispatch(**kw) == D.EINVAL, kw
    assert dispatch(x=A + 4) == D.EALIGN and dispatch(xs=A + 8) == D.EALIGN
    for kw in (dict(ys=None), dict(y=None), dict(sd=2), dict(yd=2)):
        assert combine(**kw) == D.EINVAL, kw
    for kw in (dict(ys=A + 4), dict(y=A + 4), dict(base=A + 4), dict(w=A + 2)):
        assert combine(**kw) == D.EALIGN, kw
    for kw in (dict(dy=None), dict(ys=None), dict(yd=2), dict(sd=2), dict(dys=None, dw=None, dl=None)):
        assert grad(**kw) == D.EINVAL, kw
    for kw in (dict(dy=A + 4), dict(ys=A + 4), dict(dys=A + 4), dict(w=A + 2), dict(dw=A + 2), dict(dl=A + 2)):
        assert grad(**kw) == D.EALIGN, kw


def test_mx_argument_errors():
    def quant(x=A, dt=0, T=4, inv=A, k=2, n=8, cols=256, p=A):
        return status("mx_quantize", x, dt, T, inv, k, n, cols, p, None)

    def dequant(p=A, n=8, cols=256, out=A, dt=0):
        return status("mx_dequantize", p, n, cols, out, dt, None)

    def product(a=A, n=8, cols=256, w=A, up=None, rows=16, E=4, off=A, y=A, dt=0):
        return status("mx_product", a, n, cols, w, up, rows, E, off, y, dt, None)

    def back(dy=A, dt=0, n=8, rows=16, w=A, cols=256, E=4, off=A, da=A, dd=0):
        return status("mx_product_grad", dy, dt, n, rows, w, cols, E, off, da, dd, None)

    for kw in (dict(T=0), dict(T=(1 << 20) + 1), dict(k=0), dict(k=17), dict(cols=128), dict(n=0),
               dict(n=(1 << 24) + 1), dict(inv=None), dict(inv=None, k=1, n=3)):
        assert quant(**kw) == D.ESHAPE, kw
    for kw in (dict(x=None), dict(p=None), dict(dt=5)):
        assert quant(**kw) == D.EINVAL, kw
    for kw in (dict(x=A + 8), dict(p=A + 4), dict(inv=A + 2)):
        assert quant(**kw) == D.EALIGN, kw
    for kw in (dict(n=0), dict(cols=100), dict(cols=32768)):
        assert dequant(**kw) == D.ESHAPE, kw
    for kw in (dict(p=None), dict(out=None), dict(dt=2)):
        assert dequant(**kw) == D.EINVAL, kw
    assert dequant(p=A + 4) == D.EALIGN and dequant(out=A + 4) == D.EALIGN
    for f in (product, back):
        for kw in (dict(n=0), dict(n=(1 << 24) + 1), dict(cols=128), dict(cols=16640), dict(rows=0), dict(rows=24),
                   dict(rows=16400), dict(E=0), dict(E=1025)):
            assert f(**kw) == D.ESHAPE, (f.__name__, kw)
        for kw in (dict(off=None), dict(w=None), dict(dt=2)):
            assert f(**kw) == D.EINVAL, (f.__name__, kw)
        for kw in (dict(w=A + 4), dict(off=A + 2)):
            assert f(**kw) == D.EALIGN, (f.__name__, kw)
    assert product(a=None) == D.EINVAL and product(y=None) == D.EINVAL
    assert product(a=A + 8) == D.EALIGN and product(y=A + 8) == D.EALIGN and product(up=A + 8) == D.EALIGN
    assert back(dy=None) == D.EINVAL and back(da=None) == D.EINVAL and back(dd=7) == D.EINVAL
    assert back(dy=A + 8) == D.EALIGN and back(da=A + 8) == D.EALIGN


def test_binding_refuses_host_tensors():
    """A tensor in host memory is refused by the binding, not read by a kernel."""
    t = torch.zeros(4, 256)
    i = torch.zeros(4, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        D.dispatch(t, D.DT_F32, 4, 1, 256, i, t, 4)
    with pytest.raises(ValueError):
        D.mx_quantize(t, D.DT_F32, 4, None, 1, 4, 256, t)
    with pytest.raises(ValueError):
        D.Norm(256, w_pre=torch.ones(128))
    with pytest.raises(ValueError):
        D.Norm(256, w_pre=torch.ones(256))


def test_refused_call_raises_with_its_name():
    with pytest.raises(D.Ds4moeError, match="ds4moe_dispatch") as e:
        D.dispatch(A, D.DT_F32, 0, 1, 256, A, A, 4)
    assert e.value.status == D.ESHAPE
