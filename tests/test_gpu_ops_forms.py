"""Every form of the MXFP4 product (few rows, and tiles of 64, 128 and 256
rows) in both output types, plain and SwiGLU, grouped and without offsets.
Which form a call takes depends on its sizes alone; each shape names the form
that it is meant for, and the library's kernel timer says which one ran, so
that a change of the rule cannot move the shapes to one kernel unseen.  Values
are held to the 64-bit products with the bounds of the products' own tests."""
import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D
from tests.ops_ref import close
from tests.test_gpu_ops_mx import Product

pytestmark = pytest.mark.gpu

FORM = {"few": "k_mx_rows<", "64": "k_mx_mid<1,", "128": "k_mx_mid<2,", "256": "k_mx_big<"}
# form, rows, weight rows (SwiGLU takes half of them from each matrix), cols, experts
SHAPES = [("few", 40, 288, 768, 1), ("few", 60, 96, 512, 17),
          ("64", 150, 4128, 768, 1), ("64", 700, 1056, 256, 9), ("64", 1290, 2080, 512, 5),
          ("128", 1500, 4128, 512, 1), ("128", 5000, 4096, 256, 9), ("128", 1300, 8224, 256, 11),
          ("256", 3100, 4128, 768, 1), ("256", 3000, 4096, 256, 3)]


def ran(call):
    """call()'s result and the products' kernels that it launched."""
    torch.cuda.synchronize()
    D.trace_read(reset=True)
    D.trace_enable(True)
    try:
        out = call()
    finally:
        D.trace_enable(False)
    return out, [n for n, (_, count) in D.trace_read(reset=True).items() if count and n.startswith("k_mx")]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("form,n,rows,cols,E", SHAPES)
def test_product_form(form, n, rows, cols, E, glu, kind):
    rows = rows // 2 if glu else rows
    p = Product(n, rows, cols, E, 0 if E == 1 else 3, glu)
    y, m = p.ref()
    for offsets in (True, False) if E == 1 else (True,):
        got, names = ran(lambda: p.run(kind, offsets))
        assert len(names) == 1 and names[0].startswith(FORM[form]), names
        close(got, y, m, 1, f"{form} n={n} rows={rows} cols={cols} E={E} glu={glu} {kind} offsets={offsets}")
