"""Python binding of the ds4moe C ABI (include/ds4moe.h).

Argument marshalling only: every computation runs in the HIP library
libds4moe.so built next to this file.  PyTorch tensors supply device memory
and the current stream; the C functions see plain pointers and sizes.  The
module refuses to work without the built library (no CPU fallback).
"""
from __future__ import annotations

import ctypes
import os
import sys

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libds4moe.so")

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE, EHIP, EUNSUPPORTED = 0, -1, -2, -3, -4, -5, -6
FMT_F16, FMT_CB2, FMT_Q2K, FMT_MXFP4, FMT_Q4K = 0, 1, 2, 3, 4
EXPERTS_CB2_Q2K, EXPERTS_MXFP4, EXPERTS_Q4K = 0, 1, 2
DT_F32, DT_BF16 = 0, 1
MODE_DECODE, MODE_PREFILL, MODE_ROUTE = 0, 1, 2
DECODE_MAX_T = 64
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_FULL = 0, 1, 2, 3
STATE_F32, STATE_FP8 = 0, 1


class Ds4moeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {strerror(status)} (status {status})")
        self.status = status


class LayerDesc(ctypes.Structure):
    """Mirror of ds4moe_layer."""
    _fields_ = [
        ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("d_ff", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32),
        ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
        ("sh_gate", ctypes.c_void_p), ("sh_up", ctypes.c_void_p), ("sh_down", ctypes.c_void_p),
        ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
        ("expert_fmt", ctypes.c_int32),
    ]


class HcDesc(ctypes.Structure):
    """Mirror of ds4moe_hc."""
    _fields_ = [
        ("n_streams", ctypes.c_int32), ("d_model", ctypes.c_int32), ("sinkhorn_iters", ctypes.c_int32),
        ("eps", ctypes.c_float), ("alpha_pre", ctypes.c_float), ("alpha_post", ctypes.c_float),
        ("alpha_res", ctypes.c_float), ("phi", ctypes.c_void_p), ("bias", ctypes.c_void_p),
    ]


class NormDesc(ctypes.Structure):
    """Mirror of ds4moe_norm."""
    gpu = None  # the device that the weights are known to be on
    _fields_ = [
        ("d_model", ctypes.c_int32), ("eps", ctypes.c_float), ("res_scale", ctypes.c_float), ("gate", ctypes.c_int32),
        ("w_pre", ctypes.c_void_p), ("w_post", ctypes.c_void_p), ("w_next", ctypes.c_void_p),
    ]


class ParamDesc(ctypes.Structure):
    """Mirror of ds4moe_param."""
    _fields_ = [
        ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p), ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64),
        ("weight_decay", ctypes.c_double),
    ]


class AdamWDesc(ctypes.Structure):
    """Mirror of ds4moe_adamw."""
    _fields_ = [
        ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("state", ctypes.c_int32),
        ("n_params", ctypes.c_int32), ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
        ("lr_dev", ctypes.c_void_p), ("step_dev", ctypes.c_void_p), ("run", ctypes.c_int64), ("blocks", ctypes.c_int64),
        ("kinds", ctypes.c_int64),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m bit_quantized_routed_router_amd.build_lib`")
        L = ctypes.CDLL(_LIB_PATH)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        LP = ctypes.POINTER(LayerDesc)
        L.ds4moe_packed_bytes.restype = SZ
        L.ds4moe_packed_bytes.argtypes = [I32, I64, I64]
        L.ds4moe_quantize.restype = I32
        L.ds4moe_quantize.argtypes = [I32, P, I64, I64, P, P]
        L.ds4moe_dequantize.restype = I32
        L.ds4moe_dequantize.argtypes = [I32, P, I64, I64, P, P]
        L.ds4moe_workspace_bytes.restype = SZ
        L.ds4moe_workspace_bytes.argtypes = [LP, I64, I32]
        L.ds4moe_workspace_init.restype = I32
        L.ds4moe_workspace_init.argtypes = [P, SZ, P]
        L.ds4moe_route.restype = I32
        L.ds4moe_route.argtypes = [LP, P, I32, I64, P, P, P, P, P, P, SZ, P]
        L.ds4moe_forward_decode.restype = I32
        L.ds4moe_forward_decode.argtypes = [LP, P, I32, I64, P, P, P, P, SZ, P]
        L.ds4moe_forward_decode_static.restype = I32
        L.ds4moe_forward_decode_static.argtypes = [LP, P, I32, I64, P, P, P, P]
        L.ds4moe_forward_prefill.restype = I32
        L.ds4moe_forward_prefill.argtypes = [LP, P, I32, I64, P, P, P, P, P, SZ, P]
        HP = ctypes.POINTER(HcDesc)
        L.ds4moe_hc_workspace_bytes.restype = SZ
        L.ds4moe_hc_workspace_bytes.argtypes = [HP, I64]
        L.ds4moe_hc_pre.restype = I32
        L.ds4moe_hc_pre.argtypes = [HP, P, I64, P, P, P, P, SZ, P]
        L.ds4moe_hc_post.restype = I32
        L.ds4moe_hc_post.argtypes = [HP, P, P, P, I64, P, P]
        NP, N32 = ctypes.POINTER(NormDesc), ctypes.c_int32
        L.ds4moe_norm_workspace_bytes.restype = SZ
        L.ds4moe_norm_workspace_bytes.argtypes = [NP, I64]
        L.ds4moe_group_workspace_bytes.restype = SZ
        L.ds4moe_group_workspace_bytes.argtypes = [I64, N32, N32]
        AP, F32 = ctypes.POINTER(AdamWDesc), ctypes.c_float
        for name, args in {"balance_workspace": [I64, N32, N32], "xent_workspace": [I32, I64, I64, N32, I32],
                           "adamw_workspace": [AP], "adamw_table": [P, N32]}.items():
            fn = getattr(L, f"ds4moe_{name}_bytes")
            fn.restype = SZ
            fn.argtypes = args
        for name, args in {
            "norm_pre": [NP, P, I32, I64, P, I32, P],
            "norm_post": [NP, P, I32, P, I32, P, I64, P, P, I32, P],
            "norm_pre_grad": [NP, P, I32, P, I32, P, I64, P, P, P, SZ, P],
            "norm_post_grad": [NP, P, I32, P, I32, P, I64, P, P, P, P, SZ, P],
            "group": [P, I64, N32, N32, P, P, P, P, P, SZ, P],
            "dispatch": [P, I32, I64, N32, N32, P, P, I64, P],
            "combine": [P, I32, I64, P, P, P, I64, N32, N32, P, I32, P],
            "combine_grad": [P, I32, P, I32, I64, P, P, I64, N32, N32, P, P, P, P],
            "mx_quantize": [P, I32, I64, P, N32, I64, N32, P, P],
            "mx_dequantize": [P, I64, N32, P, I32, P],
            "mx_product": [P, I64, N32, P, P, N32, N32, P, P, I32, P],
            "mx_product_grad": [P, I32, I64, N32, P, N32, N32, P, P, I32, P],
            "balance": [P, I32, I64, N32, P, N32, P, N32, P, P, P, P, SZ, P],
            "balance_grad": [P, I32, I64, N32, P, N32, P, N32, P, P, P, P, P, P],
            "xent": [P, P, I32, I64, I64, N32, F32, P, P, P, P, SZ, P],
            "xent_grad": [P, P, I32, I64, I64, N32, F32, P, P, P, P, P, P, SZ, P],
            "adamw_table": [AP, P, N32, P, SZ],
            "adamw_step": [AP, P, I64, P, P],
            "adamw_norm": [AP, P, F32, P, P, SZ, P],
        }.items():
            fn = getattr(L, "ds4moe_" + name)
            fn.restype = I32
            fn.argtypes = args
        L.ds4moe_strerror.restype = ctypes.c_char_p
        L.ds4moe_strerror.argtypes = [I32]
        L.ds4moe_trace_enable.restype = I32
        L.ds4moe_trace_enable.argtypes = [I32]
        L.ds4moe_trace_read.restype = I32
        L.ds4moe_trace_read.argtypes = [P, SZ, P, P, I32, I32]
        L.ds4moe_grid_levels.restype = None
        L.ds4moe_grid_levels.argtypes = [P]
        _lib = L
    return _lib


EXPORTS = ["ds4moe_packed_bytes", "ds4moe_quantize", "ds4moe_dequantize", "ds4moe_workspace_bytes",
           "ds4moe_workspace_init",
           "ds4moe_route", "ds4moe_forward_decode", "ds4moe_forward_decode_static", "ds4moe_forward_prefill", "ds4moe_strerror",
           "ds4moe_grid_levels", "ds4moe_trace_enable", "ds4moe_trace_read",
           "ds4moe_hc_workspace_bytes", "ds4moe_hc_pre", "ds4moe_hc_post",
           "ds4moe_norm_workspace_bytes", "ds4moe_norm_pre", "ds4moe_norm_post", "ds4moe_norm_pre_grad",
           "ds4moe_norm_post_grad", "ds4moe_group_workspace_bytes", "ds4moe_group", "ds4moe_dispatch",
           "ds4moe_combine", "ds4moe_combine_grad", "ds4moe_mx_quantize", "ds4moe_mx_dequantize",
           "ds4moe_mx_product", "ds4moe_mx_product_grad", "ds4moe_balance_workspace_bytes", "ds4moe_balance",
           "ds4moe_balance_grad", "ds4moe_xent_workspace_bytes", "ds4moe_xent", "ds4moe_xent_grad",
           "ds4moe_adamw_table_bytes", "ds4moe_adamw_table", "ds4moe_adamw_workspace_bytes", "ds4moe_adamw_step",
           "ds4moe_adamw_norm"]


def strerror(status: int) -> str:
    return lib().ds4moe_strerror(int(status)).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != OK:
        raise Ds4moeError(status, what)


def packed_bytes(fmt: int, rows: int, cols: int) -> int:
    return int(lib().ds4moe_packed_bytes(fmt, rows, cols))


def quantize(fmt: int, w, rows: int, cols: int, packed, stream=None) -> None:
    _check(lib().ds4moe_quantize(fmt, _ptr(w), rows, cols, _ptr(packed), _stream(stream)), "ds4moe_quantize")


def dequantize(fmt: int, packed, rows: int, cols: int, w, stream=None) -> None:
    _check(lib().ds4moe_dequantize(fmt, _ptr(packed), rows, cols, _ptr(w), _stream(stream)), "ds4moe_dequantize")


def workspace_bytes(desc: LayerDesc, T: int, mode: int) -> int:
    return int(lib().ds4moe_workspace_bytes(ctypes.byref(desc), T, mode))


def workspace_init(ws, nbytes: int, stream=None) -> None:
    """Zero a new workspace (required once before its first forward call)."""
    _check(lib().ds4moe_workspace_init(_ptr(ws), int(nbytes), _stream(stream)), "ds4moe_workspace_init")


def route(desc, x, x_dtype, T, topk_idx, topk_w, counts, offsets, perm, ws, ws_bytes, stream=None) -> None:
    _check(lib().ds4moe_route(ctypes.byref(desc), _ptr(x), x_dtype, T, _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
                              _ptr(offsets), _ptr(perm), _ptr(ws), ws_bytes, _stream(stream)), "ds4moe_route")


def forward_decode(desc, x, x_dtype, T, y, topk_idx_out, topk_w_out, ws, ws_bytes, stream=None) -> None:
    _check(lib().ds4moe_forward_decode(ctypes.byref(desc), _ptr(x), x_dtype, T, _ptr(y), _ptr(topk_idx_out),
                                       _ptr(topk_w_out), _ptr(ws), ws_bytes, _stream(stream)), "ds4moe_forward_decode")


STATIC_SCRATCH_BYTES = 4 << 20


def forward_decode_static(desc, x, x_dtype, T, y, topk_idx_out, topk_w_out, stream=None) -> None:
    """forward_decode on the library's own device array (no workspace)."""
    _check(lib().ds4moe_forward_decode_static(ctypes.byref(desc), _ptr(x), x_dtype, T, _ptr(y), _ptr(topk_idx_out),
                                              _ptr(topk_w_out), _stream(stream)), "ds4moe_forward_decode_static")


def forward_prefill(desc, x, x_dtype, T, y, topk_idx_out, topk_w_out, perm_out, ws, ws_bytes, stream=None) -> None:
    _check(lib().ds4moe_forward_prefill(ctypes.byref(desc), _ptr(x), x_dtype, T, _ptr(y), _ptr(topk_idx_out),
                                        _ptr(topk_w_out), _ptr(perm_out), _ptr(ws), ws_bytes, _stream(stream)),
           "ds4moe_forward_prefill")


def hc_workspace_bytes(desc: HcDesc, T: int) -> int:
    return int(lib().ds4moe_hc_workspace_bytes(ctypes.byref(desc), T))


def hc_pre(desc, X, T, coef, x_out, x_bf16, ws, ws_bytes, stream=None) -> None:
    _check(lib().ds4moe_hc_pre(ctypes.byref(desc), _ptr(X), T, _ptr(coef), _ptr(x_out), _ptr(x_bf16), _ptr(ws),
                               ws_bytes, _stream(stream)), "ds4moe_hc_pre")


def hc_post(desc, X, y, coef, T, X_out, stream=None) -> None:
    _check(lib().ds4moe_hc_post(ctypes.byref(desc), _ptr(X), _ptr(y), _ptr(coef), T, _ptr(X_out), _stream(stream)),
           "ds4moe_hc_post")


class Hc:
    """Device tensors of one hyper-connection mixer plus its ds4moe_hc
    descriptor: phi float32 [2n + n*n, n*d], bias float32 [2n + n*n] (CUDA
    tensors), alpha (pre, post, res)."""

    def __init__(self, d, phi, bias, alpha, eps=1e-6, iters=20, n=4):
        self.tensors = dict(phi=phi, bias=bias)
        self.d, self.n = d, n
        a = [float(v) for v in alpha]
        self.desc = HcDesc(n, d, iters, float(eps), a[0], a[1], a[2], _ptr(phi), _ptr(bias))

    def workspace(self, T: int):
        n = hc_workspace_bytes(self.desc, T)
        if n == 0:
            raise Ds4moeError(ESHAPE, "ds4moe_hc_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        workspace_init(ws, n)
        return ws, n


# ---------------------------------------------------------------- operators around the layer
# Norms, tokens sorted by expert and back, MXFP4 rows and products: thin calls
# of the C functions of the same names.  The library sees bare addresses, so a
# tensor's device, layout, type and size are checked here against what the
# call reads and writes (an int is taken as an address, None as NULL: those go
# unchecked).

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# what a tensor holds beside the type codes' values (bfloat16 also as its bits)
_I32, _BYTES = 100, 101
_addresses = None


def _load_addresses():
    """The native argument checks (csrc/binding/tensor_args.cpp)."""
    global _addresses
    if _addresses is None:
        try:
            from ._tensor_args import addresses
        except ImportError as e:
            raise RuntimeError("the binding's _tensor_args.so is missing or does not load: build it with "
                               "`python -m bit_quantized_routed_router_amd.build_lib`") from e
        _addresses = addresses
    return _addresses


def _call(name: str, stream, *args) -> None:
    """Run a C function, the stream last.  A tensor comes as (tensor, count,
    what it holds): it has to hold at least `count` values, or bytes.  The
    current stream's handle is taken without building the Stream object that
    torch.cuda.current_stream() returns (0.2 us against 2.8)."""
    dev = _current_gpu()
    flat = (_addresses or _load_addresses())(name, dev, args)
    flat.append(_stream(stream) if stream is not None or dev < 0 else _raw_stream(dev))
    status = getattr(_lib or lib(), name)(*flat)
    if status != OK:
        raise Ds4moeError(status, name)


def _on_gpu(desc):
    """A norm's descriptor, if its weights are on the current GPU."""
    if desc.gpu is not None and desc.gpu != _current_gpu():
        raise ValueError("the norm's weights are not on the current GPU")
    return desc


def _current_gpu() -> int:
    """The current device's index; -2, which no tensor has, before anything has used the GPU."""
    global _current_gpu
    if not torch.cuda.is_initialized():
        return -2
    _current_gpu = torch._C._cuda_getDevice  # from now on without the question
    return _current_gpu()


def _gate(desc, gate, T):
    return gate, (0, T, desc.d_model, T * desc.d_model)[desc.gate] if 0 <= desc.gate <= GATE_FULL else 0, DT_F32


def norm_workspace_bytes(desc: NormDesc, T: int) -> int:
    return int(lib().ds4moe_norm_workspace_bytes(ctypes.byref(desc), T))


def norm_pre(desc, h, h_dtype, T, x, x_dtype, stream=None) -> None:
    n = T * desc.d_model
    _call("ds4moe_norm_pre", stream, _on_gpu(desc), (h, n, h_dtype), h_dtype, T, (x, n, x_dtype), x_dtype)


def norm_post(desc, h, h_dtype, y, y_dtype, gate, T, h_out, x_next, x_dtype, stream=None) -> None:
    n = T * desc.d_model
    _call("ds4moe_norm_post", stream, _on_gpu(desc), (h, n, h_dtype), h_dtype, (y, n, y_dtype), y_dtype,
          _gate(desc, gate, T), T, (h_out, n, h_dtype), (x_next, n, x_dtype), x_dtype)


def norm_pre_grad(desc, h, h_dtype, dx, x_dtype, dh_out, T, dh, dw_pre, ws, ws_bytes, stream=None) -> None:
    n = T * desc.d_model
    _call("ds4moe_norm_pre_grad", stream, _on_gpu(desc), (h, n, h_dtype), h_dtype, (dx, n, x_dtype), x_dtype,
          (dh_out, n, h_dtype), T, (dh, n, h_dtype), (dw_pre, desc.d_model, DT_F32), (ws, ws_bytes, _BYTES), ws_bytes)


def norm_post_grad(desc, dh_out, h_dtype, y, y_dtype, gate, T, dy, dw_post, dgate, ws, ws_bytes, stream=None) -> None:
    n = T * desc.d_model
    _call("ds4moe_norm_post_grad", stream, _on_gpu(desc), (dh_out, n, h_dtype), h_dtype, (y, n, y_dtype), y_dtype,
          _gate(desc, gate, T), T, (dy, n, y_dtype), (dw_post, desc.d_model, DT_F32), _gate(desc, dgate, T),
          (ws, ws_bytes, _BYTES), ws_bytes)


class Norm:
    """Weights of a block's norms (float32 CUDA tensors [d] on one GPU, or None
    for ones) plus the ds4moe_norm descriptor."""

    def __init__(self, d, eps=1e-6, res_scale=1.0, gate=GATE_NONE, w_pre=None, w_post=None, w_next=None):
        self.tensors = dict(w_pre=w_pre, w_post=w_post, w_next=w_next)
        gpu = None
        for name, w in self.tensors.items():
            if w is None:
                continue
            if w.dtype != torch.float32 or w.numel() != d or not w.is_cuda or not w.is_contiguous():
                raise ValueError(f"{name}: expected {d} contiguous float32 values on the GPU")
            if gpu is not None and gpu != w.get_device():
                raise ValueError(f"{name}: expected the weights on one GPU")
            gpu = w.get_device()
        self.d = d
        self.desc = NormDesc(d, float(eps), float(res_scale), gate, _ptr(w_pre), _ptr(w_post), _ptr(w_next))
        self.desc.gpu = gpu

    def workspace(self, T: int):
        n = norm_workspace_bytes(self.desc, T)
        if n == 0:
            raise Ds4moeError(ESHAPE, "ds4moe_norm_workspace_bytes")
        return torch.empty(n, dtype=torch.uint8, device="cuda"), n


def group_workspace_bytes(T: int, k: int, n_experts: int) -> int:
    return int(lib().ds4moe_group_workspace_bytes(T, k, n_experts))


def group(topk_idx, T, k, n_experts, counts, offsets, perm, inv, ws, ws_bytes, stream=None) -> None:
    s = T * k
    _call("ds4moe_group", stream, (topk_idx, s, _I32), T, k, n_experts, (counts, n_experts, _I32),
          (offsets, n_experts + 1, _I32), (perm, s, _I32), (inv, s, _I32), (ws, ws_bytes, _BYTES), ws_bytes)


def dispatch(x, x_dtype, T, k, d, inv, xs, n_rows, stream=None) -> None:
    _call("ds4moe_dispatch", stream, (x, T * d, x_dtype), x_dtype, T, k, d, (inv, T * k, _I32), (xs, n_rows * d, x_dtype),
          n_rows)


def combine(ys, ys_dtype, n_rows, inv, topk_w, base, T, k, d, y, y_dtype, stream=None) -> None:
    s, n = T * k, T * d
    _call("ds4moe_combine", stream, (ys, n_rows * d, ys_dtype), ys_dtype, n_rows, (inv, s, _I32),
          (topk_w, s, DT_F32), (base, n, y_dtype), T, k, d, (y, n, y_dtype), y_dtype)


def combine_grad(dy, y_dtype, ys, ys_dtype, n_rows, inv, topk_w, T, k, d, dys, dw, dlogits, stream=None) -> None:
    s, rows = T * k, n_rows * d
    _call("ds4moe_combine_grad", stream, (dy, T * d, y_dtype), y_dtype, (ys, rows, ys_dtype), ys_dtype, n_rows,
          (inv, s, _I32), (topk_w, s, DT_F32), T, k, d, (dys, rows, ys_dtype), (dw, s, DT_F32), (dlogits, s, DT_F32))


def _mx_bytes(n, cols):
    return n * cols * 17 // 32


def mx_quantize(x, x_dtype, T, inv, k, n_rows, cols, packed, stream=None) -> None:
    _call("ds4moe_mx_quantize", stream, (x, T * cols, x_dtype), x_dtype, T, (inv, T * k, _I32), k, n_rows,
          cols, (packed, _mx_bytes(n_rows, cols), _BYTES))


def mx_dequantize(packed, n_rows, cols, out, out_dtype, stream=None) -> None:
    _call("ds4moe_mx_dequantize", stream, (packed, _mx_bytes(n_rows, cols), _BYTES), n_rows, cols,
          (out, n_rows * cols, out_dtype), out_dtype)


def mx_product(a, n_rows, cols, w, w_up, rows, n_experts, offsets, y, y_dtype, stream=None) -> None:
    m = n_experts * _mx_bytes(rows, cols)
    _call("ds4moe_mx_product", stream, (a, _mx_bytes(n_rows, cols), _BYTES), n_rows, cols, (w, m, _BYTES),
          (w_up, m, _BYTES), rows, n_experts, (offsets, n_experts + 1, _I32),
          (y, n_rows * rows, y_dtype), y_dtype)


def mx_product_grad(dy, dy_dtype, n_rows, rows, w, cols, n_experts, offsets, da, da_dtype, stream=None) -> None:
    _call("ds4moe_mx_product_grad", stream, (dy, n_rows * rows, dy_dtype), dy_dtype, n_rows, rows,
          (w, n_experts * _mx_bytes(rows, cols), _BYTES), cols, n_experts, (offsets, n_experts + 1, _I32),
          (da, n_rows * cols, da_dtype), da_dtype)


# ---------------------------------------------------------------- a training step
# The router's balance loss, the cross entropy against a vocabulary and AdamW:
# thin calls as above.

def balance_workspace_bytes(T: int, n_experts: int, n_seqs: int) -> int:
    return int(lib().ds4moe_balance_workspace_bytes(T, n_experts, n_seqs))


def balance(logits, l_dtype, T, n_experts, topk_idx, k, seq_offsets, n_seqs, counts, tokens, loss, ws, ws_bytes,
            stream=None) -> None:
    _call("ds4moe_balance", stream, (logits, T * n_experts, l_dtype), l_dtype, T, n_experts, (topk_idx, T * k, _I32), k,
          (seq_offsets, n_seqs + 1, _I32), n_seqs, (counts, n_seqs * n_experts, _I32), (tokens, n_seqs, _I32),
          (loss, n_seqs, DT_F32), (ws, ws_bytes, _BYTES), ws_bytes)


def balance_grad(logits, l_dtype, T, n_experts, topk_idx, k, seq_offsets, n_seqs, counts, tokens, dloss, dslots, dlogits,
                 stream=None) -> None:
    n = T * n_experts
    _call("ds4moe_balance_grad", stream, (logits, n, l_dtype), l_dtype, T, n_experts, (topk_idx, T * k, _I32), k,
          (seq_offsets, n_seqs + 1, _I32), n_seqs, (counts, n_seqs * n_experts, _I32), (tokens, n_seqs, _I32),
          (dloss, n_seqs, DT_F32), (dslots, T * k, DT_F32), (dlogits, n, l_dtype))


def xent_workspace_bytes(dtype: int, T: int, vocab: int, d: int, with_grad: bool) -> int:
    return int(lib().ds4moe_xent_workspace_bytes(dtype, T, vocab, d, int(with_grad)))


def xent(h, w, dtype, T, vocab, d, scale, target, loss, lse, ws, ws_bytes, stream=None) -> None:
    _call("ds4moe_xent", stream, (h, T * d, dtype), (w, vocab * d, dtype), dtype, T, vocab, d, scale, (target, T, _I32),
          (loss, T, DT_F32), (lse, T, DT_F32), (ws, ws_bytes, _BYTES), ws_bytes)


def xent_grad(h, w, dtype, T, vocab, d, scale, target, lse, dloss, dh, dw, ws, ws_bytes, stream=None) -> None:
    _call("ds4moe_xent_grad", stream, (h, T * d, dtype), (w, vocab * d, dtype), dtype, T, vocab, d, scale,
          (target, T, _I32), (lse, T, DT_F32), (dloss, T, DT_F32), (dh, T * d, dtype), (dw, vocab * d, dtype),
          (ws, ws_bytes, _BYTES), ws_bytes)


class AdamW:
    """Tensors that AdamW updates (lists of equal length, on the current GPU) plus
    the ds4moe_adamw descriptor and its table on the GPU.

    params, grads: float32 or bfloat16, one type each; master: float32, or None
    (for all, or in a tensor's place); m, v: float32, or torch.float8_e4m3fn (or
    uint8) codes with m_scale and v_scale, float32 with one value for each 256.
    weight_decay: one value, or one a tensor.  lr_dev float32 [1] and step_dev
    int32 [1] on the GPU take lr's and the step's place (for captured graphs);
    desc.lr may be set between steps.  The table holds addresses: gradients stay
    in their tensors from step to step, or set_grads writes them anew.  A captured
    step reads the table when it runs: the object has to outlive the graph.
    Otherwise it may go while steps are pending: where one was called on another
    stream than the one current at construction, which the table's memory belongs
    to, its end waits for the GPU."""

    _TYPES = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}
    _CODES = (torch.float8_e4m3fn, torch.uint8)

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None, master=None, lr=1e-3, beta1=0.9, beta2=0.999,
                 eps=1e-8, weight_decay=0.0, lr_dev=None, step_dev=None):
        import numpy as np
        fp8 = m_scale is not None or v_scale is not None
        given = dict(param=params, grad=grads, master=master, m=m, v=v, m_scale=m_scale, v_scale=v_scale)
        # (lists of its own: what the table points to stays, whatever becomes of the caller's)
        self.tensors = {name: None if ts is None else list(ts) for name, ts in given.items()}
        params, grads = self.tensors["param"], self.tensors["grad"]
        self.sizes = [p.numel() for p in params]
        self.devices = (lr_dev, step_dev)
        self.weight_decay = np.array(weight_decay, dtype=np.float64)  # (a copy, as the lists are)
        self.gpu = _current_gpu()
        # the stream that the table's memory belongs to, and whether another one may read it
        self.home, self.away = _stream(None), False
        one = lambda name, ts: self._type(name, ts[0]) if ts else DT_F32  # noqa: E731
        lr_at, step_at = self._check([(lr_dev, 1, DT_F32), (step_dev, 1, _I32)])
        self.desc = AdamWDesc(one("params", params), one("grads", grads), STATE_FP8 if fp8 else STATE_F32, 0, lr, beta1,
                              beta2, eps, lr_at, step_at, 0, 0, 0)
        self.table = None
        self._make_table(self.tensors)

    def _type(self, name, t):
        if t.dtype not in self._TYPES:
            raise ValueError(f"{name}: a tensor of dtype {t.dtype}")
        return self._TYPES[t.dtype]

    def _check(self, args):
        return (_addresses or _load_addresses())("AdamW", self.gpu, tuple(args))

    def _make_table(self, tensors):
        import numpy as np
        n, desc = len(self.sizes), self.desc
        fp8 = desc.state == STATE_FP8
        rows = np.zeros(n, dtype=[(f[0], "<i8" if f[0] == "n" else "<f8" if f[0] == "weight_decay" else "<u8")
                                  for f in ParamDesc._fields_])
        blocks = [(k + 255) // 256 for k in self.sizes]
        held = dict(param=desc.param_dtype, grad=desc.grad_dtype)
        for name, ts in tensors.items():
            scale = name.endswith("_scale")
            if ts is None and (name == "master" or scale and not fp8):
                continue
            if ts is None or len(ts) != n:
                raise ValueError(f"{name}: expected {n} tensors")
            codes = fp8 and name in ("m", "v")
            if codes and any(t.dtype not in self._CODES for t in ts):
                raise ValueError(f"{name}: codes are float8_e4m3fn or uint8")
            what = _BYTES if codes else held.get(name, DT_F32)
            at = self._check([(t, k, what) for t, k in zip(ts, blocks if scale else self.sizes)])
            rows[name] = [0 if a is None else a for a in at]
        rows["n"] = self.sizes
        rows["weight_decay"] = self.weight_decay
        size = int(lib().ds4moe_adamw_table_bytes(rows.ctypes.data, n))
        table = torch.empty(size, dtype=torch.uint8)
        _check(lib().ds4moe_adamw_table(ctypes.byref(desc), rows.ctypes.data, n, _ptr(table), size), "ds4moe_adamw_table")
        if self.table is not None:  # in place, once no step reads it any more
            torch.cuda.synchronize(self.gpu)
            self.table.copy_(table)
        elif self.gpu >= 0:
            self.table = table.cuda()

    def __del__(self):
        if getattr(self, "table", None) is None or not self.away or sys.is_finalizing():
            return
        if torch.cuda.is_current_stream_capturing():  # no waiting here: it goes with the next one
            _left.append(self.table)
        else:
            torch.cuda.synchronize(self.gpu)
            _left.clear()

    def set_grads(self, grads) -> None:
        """Gradients in other tensors, of the type they had.  The table keeps its
        place, so a captured step takes them too.  Waits for the GPU."""
        grads = list(grads)
        if grads and self._type("grads", grads[0]) != self.desc.grad_dtype:
            raise ValueError(f"grads: a tensor of dtype {grads[0].dtype} where the table has another")
        tensors = dict(self.tensors, grad=grads)
        self._make_table(tensors)
        self.tensors = tensors

    def workspace_bytes(self) -> int:
        return int(lib().ds4moe_adamw_workspace_bytes(ctypes.byref(self.desc)))


_left = []  # tables whose optimizers went during a capture


def _adamw_stream(opt, stream):
    """The call's stream, noted where the table's memory belongs to another."""
    if opt.gpu != _current_gpu():
        raise ValueError("the optimizer's tensors are not on the current GPU")
    at = _stream(stream) if stream is not None or opt.gpu < 0 else _raw_stream(opt.gpu)
    if at != opt.home:
        opt.away = True
    return at


def adamw_step(opt: AdamW, step, grad_scale=None, stream=None) -> None:
    _call("ds4moe_adamw_step", _adamw_stream(opt, stream), opt.desc, (opt.table, 1, _BYTES), step, (grad_scale, 1, DT_F32))


def adamw_norm(opt: AdamW, max_norm, out, ws, ws_bytes, stream=None) -> None:
    _call("ds4moe_adamw_norm", _adamw_stream(opt, stream), opt.desc, (opt.table, 1, _BYTES), max_norm, (out, 2, DT_F32),
          (ws, ws_bytes, _BYTES), ws_bytes)


def trace_enable(on: bool) -> None:
    lib().ds4moe_trace_enable(1 if on else 0)


def trace_read(reset: bool = True) -> dict:
    """{kernel name: (total ms, launches)} accumulated since the last reset."""
    cap = 64
    names = ctypes.create_string_buffer(8192)
    ms = (ctypes.c_double * cap)()
    cnt = (ctypes.c_longlong * cap)()
    n = lib().ds4moe_trace_read(names, 8192, ctypes.cast(ms, ctypes.c_void_p), ctypes.cast(cnt, ctypes.c_void_p),
                                cap, 1 if reset else 0)
    if n < 0:
        raise Ds4moeError(n, "ds4moe_trace_read")
    keys = names.value.decode().split("\n")[:min(n, cap)]
    return {k: (ms[i], cnt[i]) for i, k in enumerate(keys)}


def grid_levels():
    import numpy as np
    out = np.zeros((256, 8), dtype=np.uint8)
    lib().ds4moe_grid_levels(out.ctypes.data_as(ctypes.c_void_p))
    return out


class Layer:
    """Device tensors of one layer plus its ds4moe_layer descriptor.

    router_w, sh_gate, sh_up, sh_down: binary16 bit patterns (int16/uint16 or
    float16 CUDA tensors); gate/up/down: uint8 CUDA tensors of E packed
    matrices each; router_bias: float32 CUDA tensor or None; expert_fmt:
    EXPERTS_CB2_Q2K, EXPERTS_MXFP4 or EXPERTS_Q4K.
    """

    def __init__(self, d, E, k, f, fs, router_w, router_bias, sh_gate, sh_up, sh_down, gate, up, down,
                 expert_fmt=EXPERTS_CB2_Q2K):
        self.tensors = dict(router_w=router_w, router_bias=router_bias, sh_gate=sh_gate, sh_up=sh_up,
                            sh_down=sh_down, gate=gate, up=up, down=down)
        self.d, self.E, self.k, self.f, self.fs = d, E, k, f, fs
        self.expert_fmt = expert_fmt
        self.desc = LayerDesc(d, E, k, f, fs, _ptr(router_w), _ptr(router_bias), _ptr(sh_gate), _ptr(sh_up),
                              _ptr(sh_down), _ptr(gate), _ptr(up), _ptr(down), expert_fmt)

    def with_experts(self, gate, up, down) -> "Layer":
        t = dict(self.tensors)
        return Layer(self.d, self.E, self.k, self.f, self.fs, t["router_w"], t["router_bias"], t["sh_gate"],
                     t["sh_up"], t["sh_down"], gate, up, down, self.expert_fmt)

    def workspace(self, T: int, mode: int):
        n = workspace_bytes(self.desc, T, mode)
        if n == 0:
            raise Ds4moeError(ESHAPE, "ds4moe_workspace_bytes")
        ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
        workspace_init(ws, n)
        return ws, n
