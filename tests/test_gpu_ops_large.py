"""The operators around the layer at sizes whose grids or counts pass 32 bits.
Each result is compared with the same rows handled by a short call."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D

pytestmark = pytest.mark.gpu

BF = D.DT_BF16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_dequantize_more_than_2_to_the_35_values():
    """18 GB of packed rows to 69 GB: more threads than one launch takes."""
    n, cols = (1 << 23) + 3, 4096
    codes, scales = n * cols // 2, n * cols // 32
    packed = torch.empty(codes + scales, dtype=torch.uint8, device="cuda")
    packed.random_(0, 256, generator=gen(1))
    out = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
    out.view(torch.int16).fill_(0x1234)
    D.mx_dequantize(packed, n, cols, out, BF)
    few = torch.empty(64, cols, dtype=torch.bfloat16, device="cuda")
    for lo in (0, (1 << 22) - 40, (1 << 22), (1 << 23) - 61, n - 64):
        part = torch.cat([packed[lo * cols // 2:(lo + 64) * cols // 2],
                          packed[codes + lo * cols // 32:codes + (lo + 64) * cols // 32]])
        D.mx_dequantize(part, 64, cols, few, BF)
        assert torch.equal(out[lo:lo + 64].view(torch.int16), few.view(torch.int16)), lo


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_quantize_more_rows_than_a_sorted_call_has_tokens(kind):
    """Row by row: the hidden rows of six slots a token pass 2^20 long before
    their tokens do."""
    n, cols = (2 << 20) + 70, 256
    x = torch.randn(n, cols, dtype=kind, device="cuda", generator=gen(2))
    packed = torch.full((n * cols * 17 // 32,), 0xA5, dtype=torch.uint8, device="cuda")
    dt = BF if kind == torch.bfloat16 else D.DT_F32
    D.mx_quantize(x, dt, n, None, 1, n, cols, packed)
    ref = torch.empty_like(packed)
    D.quantize(D.FMT_MXFP4, x.float(), n, cols, ref)
    assert torch.equal(packed, ref)
