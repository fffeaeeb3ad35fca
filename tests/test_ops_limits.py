"""Sizes that the operators around the layer take and refuse, where a limit is
not that of another call's (no device work: what passes the size checks is
stopped by its alignment)."""
from bit_quantized_routed_router_amd import ds4moe as D

A = 0x10000  # stand-in device address: aligned, never dereferenced


def test_quantize_row_by_row_takes_as_many_rows_as_a_matrix_has():
    def quant(T, inv=None, k=1, n=1 << 24):
        return D.lib().ds4moe_mx_quantize(A, 0, T, inv, k, n, 256, A + 4, None)

    for T in ((1 << 20) + 1, 1 << 24):
        assert quant(T) == D.EALIGN, T
        assert quant(T, inv=A) == D.ESHAPE, T
    for T in (0, -1, (1 << 24) + 1):
        assert quant(T) == D.ESHAPE, T
    assert quant(1 << 20, inv=A, k=16) == D.EALIGN
    assert quant(4, inv=A, k=17) == D.ESHAPE and quant(4, k=2) == D.ESHAPE and quant(9, n=8) == D.ESHAPE


def test_product_gradient_refuses_more_values_than_a_launch_covers():
    def back(n, cols, dt=0):
        return D.lib().ds4moe_mx_product_grad(A, dt, n, 16, A, cols, 1, None, A + 4, 0, None)

    for dt in (D.DT_F32, D.DT_BF16):
        for n, cols in ((1 << 24, 8192), (1 << 24, 16384), (1 << 23, 16384), ((1 << 24) - 32768, 8192)):
            assert back(n, cols, dt) == (D.ESHAPE if n * cols > 2 ** 37 - 2 ** 29 else D.EALIGN), (n, cols)
        assert back((1 << 24) - 65536, 8192, dt) == D.EALIGN
