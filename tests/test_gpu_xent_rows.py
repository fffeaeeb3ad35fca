"""Softmax cross entropy of thousands of rows (live ones are found in one launch
up to 2048), rows without a target among them, and 256 x 256 tiles over several
chunks."""
import pytest
import torch

from tests import train_ref as R
from tests.test_gpu_xent import check, make, run

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rows without a target
@pytest.mark.parametrize("kind,T", [("f32", 400), ("f32", 2100), ("bf16", 2100)])
def test_rows_without_a_target_hide_what_they_hold(kind, T):
    h, w, y, dloss = make(T, 200, 256, kind, seed=14)
    y[::3] = -100
    y[1::41] = 200
    live = (y >= 0) & (y < 200)
    want = run(h, w, y, 1.0, dloss)
    h2, d2 = h.clone(), dloss.clone()
    h2[~live] = float("nan")
    h2[3] = float("inf")
    d2[~live] = float("nan")
    got = run(h2, w, y, 1.0, d2)
    for name in ("dh", "dw", "loss"):
        assert torch.equal(got[name], want[name]), name
    assert torch.equal(got["lse"][live], want["lse"][live])
    assert (got["dh"][~live] == 0).all() and (got["loss"][~live] == 0).all()


@pytest.mark.parametrize("kind,T", [("f32", 400), ("f32", 2100), ("bf16", 2100)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_rows_stay_apart(bad, kind, T):
    h, w, y, dloss = make(T, 150, 256, kind, seed=15, dead=0.2)
    y[5] = 7
    want = run(h, w, y, 1.0, dloss)
    h[5, 7] = bad
    got = run(h, w, y, 1.0, dloss)
    others = torch.arange(T) != 5
    for name in ("loss", "lse", "dh"):
        assert torch.equal(got[name][others], want[name][others]), name
        assert not torch.isfinite(got[name][5]).any(), name


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2049, 2100, 4099])
@pytest.mark.parametrize("dead", [0.0, 0.3, 0.9])
def test_thousands_of_rows(T, dead, kind):
    h, w, y, dloss = make(T, 90, 256, kind, seed=16, dead=dead)
    check(h, w, y, 1.0, dloss, f"{T} rows, {dead} without a target, {kind}")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_thousands_of_rows_and_none_or_one_with_a_target(kind):
    h, w, y, dloss = make(2500, 60, 256, kind, seed=17)
    none = run(h, w, torch.full_like(y, -1), 1.0, dloss)
    assert (none["loss"] == 0).all() and (none["dh"] == 0).all() and (none["dw"] == 0).all()
    for at in (0, 1023, 1024, 2499):
        one = torch.full_like(y, -1)
        one[at] = y[at]
        check(h, w, one, 1.0, dloss, f"row {at} alone")


# ---------------------------------------------------------------- 256 x 256 tiles over several chunks
def heavy(T, every):
    """Upstream gradients of which one row in `every` counts: a sum over rows is
    then of a few terms, and its bound close to their rounding."""
    dloss = torch.full((T,), 2.0 ** -14)
    dloss[::every] = 1 + torch.arange(len(dloss[::every])) / 8
    return dloss


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [450, 2049])
def test_large_tiles_of_dw(T, kind):
    """17 x 8 tiles of 256 x 256, rows in chunks of 64, the last one part filled.
    Rows are small, so that the logits' own rounding is nothing."""
    h, w, y, _ = make(T, 4352 - 100, 2048, kind, seed=18, dead=0.1)
    h = h * 2.0 ** -14
    dloss = heavy(T, 60 if T < 1000 else 300)
    got = run(h, w, y, 1.0, dloss, want=("dw",))
    ref = R.Xent(h, w, y, 1.0, dloss)
    R.within(got["dw"], ref.dw, ref.edw, "dw")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_large_tiles_of_logits(kind):
    """17 x 9 tiles of 256 x 256 for the sums and for ds, four chunks each, rows
    without a target between them."""
    h, w, y, dloss = make(2200, 4352 - 3, 256, kind, seed=19, dead=0.1)
    check(h, w, y, 1.0, dloss, kind)
