"""What the binding of the operators around the layer checks of the tensors it
is given: their type against the type code, their size against what the call
reads and writes, their device.  The library sees bare addresses, so a tensor
that is too short or of another type would be read or written past its end.
The refusals are shown on host tensors: type and size are looked at before the
device."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D

T, K, E, DIM, N, ROWS, COLS = 4, 2, 3, 256, 8, 32, 512
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
FLOATS = ((F32, D.DT_F32), (BF16, D.DT_BF16))


def mx(n, cols):
    return n * cols * 17 // 32


def calls(a, b):
    """name -> (function, arguments) with tensors as (count, dtype); a, b: two
    (dtype, code) pairs."""
    (at, ac), (bt, bc) = a, b
    x, row = (T * DIM, at), (N * DIM, bt)
    idx, f32 = (T * K, I32), (T * K, F32)
    out = {
        "norm_pre": (D.norm_pre, ["desc", x, ac, T, (T * DIM, bt), bc]),
        "norm_post": (D.norm_post, ["desc", x, ac, (T * DIM, bt), bc, (T * DIM, F32), T, x, (T * DIM, bt), bc]),
        "norm_pre_grad": (D.norm_pre_grad, ["desc", x, ac, (T * DIM, bt), bc, x, T, x, (DIM, F32), (4096, U8), 4096]),
        "norm_post_grad": (D.norm_post_grad, ["desc", x, ac, (T * DIM, bt), bc, (T * DIM, F32), T, (T * DIM, bt),
                                              (DIM, F32), (T * DIM, F32), (4096, U8), 4096]),
        "group": (D.group, [idx, T, K, E, (E, I32), (E + 1, I32), idx, idx, (256, U8), 256]),
        "dispatch": (D.dispatch, [x, ac, T, K, DIM, idx, (N * DIM, at), N]),
        "combine": (D.combine, [row, bc, N, idx, f32, x, T, K, DIM, x, ac]),
        "combine_grad": (D.combine_grad, [x, ac, row, bc, N, idx, f32, T, K, DIM, row, f32, f32]),
        "mx_quantize": (D.mx_quantize, [(T * COLS, at), ac, T, idx, K, N, COLS, (mx(N, COLS), U8)]),
        "mx_dequantize": (D.mx_dequantize, [(mx(N, COLS), U8), N, COLS, (N * COLS, at), ac]),
        "mx_product": (D.mx_product, [(mx(N, COLS), U8), N, COLS, (E * mx(ROWS, COLS), U8), (E * mx(ROWS, COLS), U8), ROWS,
                                      E, (E + 1, I32), (N * ROWS, at), ac]),
        "mx_product_grad": (D.mx_product_grad, [(N * ROWS, at), ac, N, ROWS, (E * mx(ROWS, COLS), U8), COLS, E,
                                                (E + 1, I32), (N * COLS, bt), bc]),
    }
    return out


NAMES = list(calls(FLOATS[0], FLOATS[0]))


def make(args, device, change=None, to=None):
    """Arguments with their tensors made; argument `change` as to(count, dtype).
    Without a device the others are stand-in addresses, which go unchecked."""
    out = []
    for i, v in enumerate(args):
        if isinstance(v, str):
            v = D.NormDesc(DIM, 1e-6, 1.0, D.GATE_FULL, None, None, None)
        elif isinstance(v, tuple):
            n, t = to(*v) if i == change else v
            v = 0x10000 if device is None and i != change else torch.zeros(n, dtype=t, device=device)
        out.append(v)
    return out


@pytest.mark.parametrize("a", FLOATS)
@pytest.mark.parametrize("b", FLOATS)
@pytest.mark.parametrize("name", NAMES)
def test_refused_tensors(name, a, b):
    f, args = calls(a, b)[name]
    other = {F32: (BF16, torch.float16, torch.float64, I32), BF16: (F32, torch.float16, U8),
             I32: (torch.int64, torch.int16, F32)}
    for i, v in enumerate(args):
        if not isinstance(v, tuple):
            continue
        with pytest.raises(ValueError, match="current GPU"):
            f(*make(args, None, i, lambda n, t: (n, t)))
        with pytest.raises(ValueError, match="bytes where" if v[1] == U8 else "values where"):
            f(*make(args, None, i, lambda n, t: (n - 1, t)))
        for t in other.get(v[1], ()):
            # twice as many, so that bytes would be enough
            with pytest.raises(ValueError, match="dtype"):
                f(*make(args, None, i, lambda n, _: (2 * n, t)))


def test_norm_of_another_device_is_refused():
    desc = D.NormDesc(DIM, 1e-6, 1.0, D.GATE_NONE, None, None, None)
    assert desc.gpu is None
    desc.gpu = 63
    with pytest.raises(ValueError, match="weights are not"):
        D.norm_pre(desc, 0x10000, 0, T, 0x10000, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("a", FLOATS)
@pytest.mark.parametrize("name", NAMES)
def test_accepted_tensors(name, a):
    """The same calls on the GPU: with tensors of the size that is taken, with
    longer ones, and with bfloat16 given as its bits."""
    f, args = calls(a, a)[name]
    if name.startswith("norm") and name.endswith("grad"):
        need = D.norm_workspace_bytes(D.NormDesc(DIM, 1e-6, 1.0, D.GATE_FULL, None, None, None), T)
        args[-2:] = [(need, U8), need]
    if name == "group":
        need = D.group_workspace_bytes(T, K, E)
        args[-2:] = [(need, U8), need]
    f(*make(args, "cuda"))
    for i, v in enumerate(args):
        if isinstance(v, tuple):
            f(*make(args, "cuda", i, lambda n, t: (2 * n + 8, t)))
            if v[1] == BF16:
                f(*make(args, "cuda", i, lambda n, t: (n, torch.int16)))
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_norm_knows_its_device():
    w = torch.ones(DIM, device="cuda")
    assert D.Norm(DIM, w_pre=w).desc.gpu == w.get_device() and D.Norm(DIM).desc.gpu is None
