"""The MXFP4 product gradient of very small fp32 rows.  A value goes in as
three bfloat16 parts of eight significant bits; the last bit of an fp32 value
of 2^-110 is 2^-133, bfloat16's smallest number, so larger values are held
exactly and smaller ones to less than 2^-133.  Beside that a sum takes 2 half
steps for each of its three terms a row, as in the gradient's own tests."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests.ops_ref import close, gen, mx_pack, mx_quantize, mx_values, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lo,hi", [(-110, -100), (-126, -111), (-149, -127)])
def test_product_grad_of_small_fp32_rows(lo, hi):
    n, rows, cols = 33, 96, 512
    g = gen(-lo)
    code, sc = mx_quantize(rand(g, rows, cols))
    sc = sc + 70  # weights near 2^70, so that the sums are normal numbers
    w, w64 = mx_pack(code, sc), mx_values(code, sc)
    # 24 significant bits, as far as fp32 has them there
    mant = torch.randint(2 ** 23, 2 ** 24, (n, rows), generator=g).double() * 2.0 ** -23
    sign = torch.randint(0, 2, (n, rows), generator=g).double() * 2 - 1
    dy = (sign * mant * torch.exp2(torch.randint(lo, hi + 1, (n, rows), generator=g).double())).float()
    da = torch.full((n, cols), 55.0, device="cuda")
    D.mx_product_grad(dy.cuda(), D.DT_F32, n, rows, w.cuda(), cols, 1, None, da, D.DT_F32)
    got, ref, mag = da.cpu(), dy.double() @ w64, dy.double().abs() @ w64.abs()
    lost = (dy.abs() < 2.0 ** -110).double() @ w64.abs() * 2.0 ** -133
    # what may be lost, as the roundings that close() counts
    close(got, ref, 6 * rows * mag + lost * 2.0 ** 24, 1, f"2^{lo} .. 2^{hi}")
