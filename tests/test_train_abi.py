"""Host-side checks of a training step's operators (no device work): sizes of
workspaces, and calls that are refused before anything is launched."""
import ctypes

import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D

A = 0x10000  # stand-in device address: aligned, never dereferenced
BIG = 1 << 60
NAN, INF = float("nan"), float("inf")


def status(name, *args):
    return getattr(D.lib(), "ds4moe_" + name)(*args)


# ---------------------------------------------------------------- balance
def balance(z=A, dt=0, T=8, E=16, idx=A, k=2, off=None, B=1, counts=A, tokens=A, loss=A, ws=A, nb=BIG):
    return status("balance", z, dt, T, E, idx, k, off, B, counts, tokens, loss, ws, nb, None)


def balance_grad(z=A, dt=0, T=8, E=16, idx=A, k=2, off=None, B=1, counts=A, tokens=A, dloss=None, ds=None, dz=A):
    return status("balance_grad", z, dt, T, E, idx, k, off, B, counts, tokens, dloss, ds, dz, None)


def test_balance_errors():
    for call in (balance, balance_grad):
        for kw in (dict(T=0), dict(T=-1), dict(T=(1 << 20) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(B=0),
                   dict(B=16385), dict(T=1 << 20, E=1024, B=1 << 15)):
            assert call(**kw) == D.ESHAPE, kw
        for kw in (dict(z=None), dict(idx=None), dict(counts=None), dict(tokens=None), dict(dt=2), dict(dt=-1), dict(B=2)):
            assert call(**kw) == D.EINVAL, kw
        for kw in (dict(z=A + 2), dict(z=A + 1, dt=1), dict(idx=A + 2), dict(off=A + 1), dict(counts=A + 2),
                   dict(tokens=A + 2)):
            assert call(**kw) == D.EALIGN, kw
    assert balance(loss=None) == D.EINVAL and balance(ws=None) == D.EINVAL and balance_grad(dz=None) == D.EINVAL
    for kw in (dict(loss=A + 2), dict(ws=A + 128)):
        assert balance(**kw) == D.EALIGN
    for kw in (dict(dz=A + 2), dict(dloss=A + 2), dict(ds=A + 2)):
        assert balance_grad(**kw) == D.EALIGN
    need = D.balance_workspace_bytes(1000, 16, 3)
    assert need > 0 and balance(T=1000, off=A, B=3, nb=need - 1) == D.EWORKSPACE
    for bad in ((0, 16, 1), (8, 0, 1), (8, 16, 0), (8, 2000, 1), (1 << 21, 4, 1), (8, 16, 1 << 15)):
        assert D.balance_workspace_bytes(*bad) == 0


# ---------------------------------------------------------------- cross entropy
def xent(h=A, w=A, dt=1, T=8, V=100, d=256, scale=1.0, y=A, loss=A, lse=A, ws=A, nb=BIG):
    return status("xent", h, w, dt, T, V, d, scale, y, loss, lse, ws, nb, None)


def xent_grad(h=A, w=A, dt=1, T=8, V=100, d=256, scale=1.0, y=A, lse=A, dloss=None, dh=A, dw=A, ws=A, nb=BIG):
    return status("xent_grad", h, w, dt, T, V, d, scale, y, lse, dloss, dh, dw, ws, nb, None)


def test_xent_errors():
    for call in (xent, xent_grad):
        for kw in (dict(T=0), dict(T=(1 << 20) + 1), dict(V=0), dict(V=(1 << 20) + 1), dict(d=0), dict(d=300),
                   dict(d=16640)):
            assert call(**kw) == D.ESHAPE, kw
        for kw in (dict(h=None), dict(w=None), dict(y=None), dict(lse=None), dict(ws=None), dict(dt=2), dict(scale=NAN),
                   dict(scale=INF)):
            assert call(**kw) == D.EINVAL, kw
        for kw in (dict(h=A + 8), dict(w=A + 8), dict(y=A + 2), dict(lse=A + 2), dict(ws=A + 128)):
            assert call(**kw) == D.EALIGN, kw
    assert xent(loss=None) == D.EINVAL and xent(loss=A + 2) == D.EALIGN
    assert xent_grad(dh=None, dw=None) == D.EINVAL
    for kw in (dict(dh=A + 8), dict(dw=A + 4), dict(dloss=A + 1)):
        assert xent_grad(**kw) == D.EALIGN
    for dt in (0, 1):
        need, more = D.xent_workspace_bytes(dt, 100, 5000, 512, False), D.xent_workspace_bytes(dt, 100, 5000, 512, True)
        assert 0 < need <= more
        assert xent(dt=dt, T=100, V=5000, d=512, nb=need - 1) == D.EWORKSPACE
    assert xent_grad(T=100, V=5000, d=512, nb=1024) == D.EWORKSPACE
    for bad in ((2, 8, 100, 256), (1, 0, 100, 256), (1, 8, 0, 256), (1, 8, 100, 100), (1, 1 << 21, 100, 256)):
        assert D.xent_workspace_bytes(*bad, True) == 0


def test_xent_workspace_does_not_hold_the_logits():
    """It grows with the vocabulary up to the size of a piece and of the forward
    pass's partial sums, 256 MB each; the logits have 32 GB here."""
    for dt in (0, 1):
        small, large = (D.xent_workspace_bytes(dt, 8192, V, 1024, True) for V in (1 << 17, 1 << 20))
        assert large <= small + (1 << 28) and large < (1 << 30)


# ---------------------------------------------------------------- AdamW
FAR = 1 << 44  # between stand-in addresses that a step would write


def param(i=0, **kw):
    v = dict(param=A + 6 * i * FAR, grad=A + (6 * i + 5) * FAR, master=None, m=A + (6 * i + 1) * FAR, v=A + (6 * i + 2) * FAR,
             m_scale=A + (6 * i + 3) * FAR, v_scale=A + (6 * i + 4) * FAR, n=100, weight_decay=0.1)
    v.update(kw)
    return D.ParamDesc(*(v[f[0]] for f in D.ParamDesc._fields_))


def opts(**kw):
    v = dict(param_dtype=0, grad_dtype=0, state=0, n_params=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, lr_dev=None,
             step_dev=None, run=4096, blocks=1, kinds=None)
    v.update(kw)
    if v["kinds"] is None:
        v["kinds"] = 8 | (v["param_dtype"] & 1) | (v["grad_dtype"] & 1) << 1 | (v["state"] & 1) << 2
    return D.AdamWDesc(*(v[f[0]] for f in D.AdamWDesc._fields_))


def table(o=None, p=None, n=1, to=True, nb=1 << 16):
    o = opts() if o is None else o
    ps = (D.ParamDesc * 2)(param() if p is None else p, param(n=0, param=None, grad=None, m=None, v=None))
    buf = ctypes.create_string_buffer(1 << 16)
    return status("adamw_table", ctypes.byref(o) if o else None, ctypes.addressof(ps), n, ctypes.addressof(buf) if to else None,
                  nb)


def step(o=None, t=A, at=1, scale=None):
    return status("adamw_step", ctypes.byref(opts() if o is None else o), t, at, scale, None)


def norm(o=None, t=A, most=1.0, out=A, ws=A, nb=BIG):
    return status("adamw_norm", ctypes.byref(opts() if o is None else o), t, most, out, ws, nb, None)


def test_adamw_option_errors():
    for kw in (dict(param_dtype=2), dict(grad_dtype=-1), dict(state=2), dict(lr=NAN), dict(lr=INF), dict(beta1=1.0),
               dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=NAN), dict(eps=0.0), dict(eps=NAN), dict(eps=INF),
               dict(eps=1e-60)):
        assert table(o=opts(**kw)) == step(o=opts(**kw)) == norm(o=opts(**kw)) == D.EINVAL, kw
    for kw in (dict(lr_dev=A + 2), dict(step_dev=A + 2)):
        assert table(o=opts(**kw)) == step(o=opts(**kw)) == D.EALIGN
    for name, args in (("table", (0, 0, A, BIG)), ("step", (A, 1, None, None)), ("norm", (A, 1.0, A, A, BIG, None))):
        assert status("adamw_" + name, None, *args) == D.EINVAL


def test_adamw_eps_is_a_normal_number():
    """The reciprocal of a smaller one is infinite, and zero times it NaN."""
    for eps in (2.0 ** -127, 1e-39, 1e-45):
        o = opts(eps=eps)
        assert table(o=o) == step(o=o) == norm(o=o) == D.EINVAL, eps
    assert table(o=opts(eps=2.0 ** -126)) == D.OK


def test_adamw_table_errors():
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(weight_decay=NAN)):
        assert table(p=param(**kw)) == D.EINVAL, kw
    for kw in (dict(n=-1), dict(n=(1 << 40) + 1)):
        assert table(p=param(**kw)) == D.ESHAPE
        ps = (D.ParamDesc * 1)(param(**kw))
        assert D.lib().ds4moe_adamw_table_bytes(ctypes.addressof(ps), 1) == 0
    for kw in (dict(param=A + 2), dict(grad=A + 2), dict(m=A + 2), dict(v=A + 1), dict(master=A + 2)):
        assert table(p=param(**kw)) == D.EALIGN, kw
    assert table(o=opts(param_dtype=1), p=param(param=A + 1)) == D.EALIGN
    fp8 = opts(state=D.STATE_FP8)
    for kw in (dict(m_scale=None), dict(v_scale=None)):
        assert table(o=fp8, p=param(**kw)) == D.EINVAL
        assert table(p=param(**kw)) == D.OK
    assert table(o=fp8, p=param(m_scale=A + 2, m=A + 1)) == D.EALIGN and table(o=fp8, p=param(m=A + FAR + 1)) == D.OK
    assert table(n=-1) == D.ESHAPE and table(n=0) == D.OK and table(n=2) == D.OK
    assert table(to=False) == D.EINVAL and table(nb=8) == D.EWORKSPACE
    assert D.lib().ds4moe_adamw_table_bytes(None, 1) == 0


def test_adamw_table_covers_every_value_once():
    sizes = [1, 4096, 4097, 0, 100000]
    ps = (D.ParamDesc * 5)(*(param(i, n=n) for i, n in enumerate(sizes)))
    o = opts()
    nb = D.lib().ds4moe_adamw_table_bytes(ctypes.addressof(ps), 5)
    buf = ctypes.create_string_buffer(nb)
    assert status("adamw_table", ctypes.byref(o), ctypes.addressof(ps), 5, ctypes.addressof(buf), nb) == D.OK
    assert o.n_params == 5 and o.run == 4096 and o.blocks == sum(-(-n // 4096) for n in sizes)
    assert buf.raw[:72 * 5] == bytes(ps)
    at = (72 * 5 + 15) // 16 * 16
    pairs = [tuple(int.from_bytes(buf.raw[at + 8 * i + 4 * j:at + 8 * i + 4 * j + 4], "little") for j in (0, 1))
             for i in range(o.blocks)]
    assert pairs == [(i, r) for i, n in enumerate(sizes) for r in range(-(-n // 4096))]
    # few blocks however long the tensors are
    ps = (D.ParamDesc * 3)(*(param(i, n=n) for i, n in enumerate((1 << 38, 5, 1 << 30))))
    nb = D.lib().ds4moe_adamw_table_bytes(ctypes.addressof(ps), 3)
    buf = ctypes.create_string_buffer(nb)
    assert status("adamw_table", ctypes.byref(o), ctypes.addressof(ps), 3, ctypes.addressof(buf), nb) == D.OK
    assert o.run % 4096 == 0 and o.blocks <= (1 << 17) + 3 and o.blocks * o.run >= (1 << 38) + (1 << 30)


def test_adamw_table_refuses_tensors_that_overlap():
    def both(a, b, o=None):
        ps = (D.ParamDesc * 2)(a, b)
        buf = ctypes.create_string_buffer(4096)
        return status("adamw_table", ctypes.byref(o or opts()), ctypes.addressof(ps), 2, ctypes.addressof(buf), 4096)

    a = param(0)
    assert both(a, param(1)) == D.OK
    assert both(a, a) == D.EINVAL  # a tensor twice
    for kw in (dict(param=a.param + 396), dict(m=a.v), dict(v=a.param - 396), dict(master=a.m)):
        assert both(a, param(1, **kw)) == D.EINVAL, kw
    # side by side, or read alone, is no overlap
    for kw in (dict(param=a.param + 400), dict(grad=a.grad), dict(grad=a.param + 400), dict(m_scale=a.m_scale), dict(n=0, param=a.param)):
        assert both(a, param(1, **kw)) == D.OK, kw
    assert both(a, param(1, m_scale=a.m_scale), opts(state=D.STATE_FP8)) == D.EINVAL
    assert table(p=param(master=A)) == D.EINVAL  # its own
    # a gradient that a step would change: its own values', another tensor's
    for kw in (dict(grad=a.param), dict(grad=a.m + 4)):
        assert table(p=param(0, **kw)) == both(a, param(1, **kw)) == both(param(1, **kw), a) == D.EINVAL, kw
    # one that begins before it and ends behind it
    assert both(a, param(1, n=100000, grad=a.param - 400)) == D.EINVAL


def test_a_table_is_for_its_types():
    for kw in (dict(param_dtype=1), dict(grad_dtype=1), dict(state=1)):
        o = opts(**kw)
        o.kinds = 8
        assert step(o=o) == norm(o=o) == D.EINVAL, kw


def test_adamw_step_and_norm_errors():
    for call in (step, norm):
        for kw in (dict(n_params=-1), dict(n_params=(1 << 20) + 1), dict(blocks=-1), dict(blocks=1 << 30), dict(run=0),
                   dict(run=300)):
            assert call(o=opts(**kw)) == D.ESHAPE, kw
        assert call(t=None) == D.EINVAL and call(t=A + 8) == D.EALIGN
    assert step(at=0) == D.EINVAL and step(at=-3) == D.EINVAL and step(scale=A + 2) == D.EALIGN
    for kw in (dict(most=0.0), dict(most=-1.0), dict(most=NAN), dict(out=None), dict(ws=None)):
        assert norm(**kw) == D.EINVAL, kw
    assert norm(out=A + 2) == D.EALIGN and norm(ws=A + 64) == D.EALIGN
    o = opts(blocks=100000)
    need = D.lib().ds4moe_adamw_workspace_bytes(ctypes.byref(o))
    assert need > 0 and norm(o=o, nb=need - 1) == D.EWORKSPACE
    assert D.lib().ds4moe_adamw_workspace_bytes(None) == 0
    # nothing to do launches nothing
    assert step(o=opts(n_params=0, blocks=0)) == D.OK


def test_struct_sizes():
    """The structures as the header lays them out on a 64-bit host."""
    assert ctypes.sizeof(D.ParamDesc) == 72 and ctypes.sizeof(D.AdamWDesc) == 88


# ---------------------------------------------------------------- binding
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def calls(dt, code):
    T, E, K, B, V, d = 4, 8, 2, 3, 10, 256
    return {
        "balance": (D.balance, [(T * E, dt), code, T, E, (T * K, I32), K, (B + 1, I32), B, (B * E, I32), (B, I32), (B, F32),
                                (512, U8), 512]),
        "balance_grad": (D.balance_grad, [(T * E, dt), code, T, E, (T * K, I32), K, (B + 1, I32), B, (B * E, I32), (B, I32),
                                          (B, F32), (T * K, F32), (T * E, dt)]),
        "xent": (D.xent, [(T * d, dt), (V * d, dt), code, T, V, d, 1.0, (T, I32), (T, F32), (T, F32), (512, U8), 512]),
        "xent_grad": (D.xent_grad, [(T * d, dt), (V * d, dt), code, T, V, d, 1.0, (T, I32), (T, F32), (T, F32), (T * d, dt),
                                    (V * d, dt), (512, U8), 512]),
    }


@pytest.mark.parametrize("dt,code", [(F32, 0), (BF16, 1)])
@pytest.mark.parametrize("name", ["balance", "balance_grad", "xent", "xent_grad"])
def test_refused_tensors(name, dt, code):
    f, args = calls(dt, code)[name]
    for i, a in enumerate(args):
        if not isinstance(a, tuple):
            continue
        for n, t, match in ((a[0], a[1], "current GPU"), (a[0] - 1, a[1], "bytes where" if a[1] == U8 else "values where"),
                            (2 * a[0], torch.float64, "bytes|dtype|current GPU" if a[1] == U8 else "dtype")):
            given = [torch.zeros(n, dtype=t) if j == i else A if isinstance(b, tuple) else b for j, b in enumerate(args)]
            with pytest.raises(ValueError, match=match):
                f(*given)


def test_optimizer_refuses_what_a_step_cannot_take():
    """Lists that do not match, types, and tensors that are not on the GPU."""
    t = [torch.zeros(300)]
    with pytest.raises(ValueError, match="current GPU"):
        D.AdamW(t, t, t, t)
    with pytest.raises(ValueError, match="grad: expected 0 tensors"):
        D.AdamW([], t, [], [])
    for bad in (torch.float16, torch.int32):
        with pytest.raises(ValueError, match="dtype"):
            D.AdamW([t[0].to(bad)], t, t, t)
    with pytest.raises(ValueError, match="v_scale: expected 0 tensors"):
        D.AdamW([], [], [], [], m_scale=[])
    with pytest.raises(ValueError, match="dtype|current GPU"):
        D.AdamW([], [], [], [], lr_dev=torch.zeros(1, dtype=torch.float64))
    assert D.AdamW([], [], [], []).desc.blocks == 0


def test_refused_gradients_leave_the_optimizer_as_it_was():
    opt = D.AdamW([], [], [], [])
    t = [torch.zeros(300)]
    with pytest.raises(ValueError, match="grad: expected 0 tensors"):
        opt.set_grads(t)
    with pytest.raises(ValueError, match="dtype"):
        opt.set_grads([t[0].bfloat16()])
    assert opt.tensors["grad"] == [] and opt.desc.grad_dtype == D.DT_F32


def test_the_optimizer_keeps_lists_of_its_own():
    given = []
    opt = D.AdamW(given, given, given, given)
    given.append(torch.zeros(3))
    assert opt.tensors["param"] == opt.tensors["grad"] == opt.tensors["m"] == opt.tensors["v"] == []


def test_optimizer_of_another_device_is_refused():
    opt = D.AdamW([], [], [], [])
    opt.gpu = 63
    with pytest.raises(ValueError, match="optimizer's tensors are not"):
        D.adamw_step(opt, 1)
