"""The optimizer's table, which is the binding's own memory, outlives the steps
that read it."""
import gc

import pytest
import torch

from bit_quantized_routed_router_amd import ds4moe as D

pytestmark = pytest.mark.gpu
N = 4097


def tensors(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = {n: torch.randn(N, generator=g, device="cuda") for n in ("p", "g", "m")}
    t["v"] = torch.rand(N, generator=g, device="cuda")
    return t


def optimizer(t):
    return D.AdamW([t["p"]], [t["g"]], [t["m"]], [t["v"]])


def busy(stream):
    """Some milliseconds of work on a stream, before what comes next on it."""
    with torch.cuda.stream(stream):
        a = torch.randn(4096, 4096, device="cuda")
        for _ in range(40):
            a = torch.mm(a, a).clamp_(-1, 1)
    return a


@pytest.mark.parametrize("call", ["given", "current"])
def test_an_optimizer_that_goes_while_a_step_on_another_stream_is_pending(call):
    """Its table's place is handed out no earlier than the step is done."""
    t, want = tensors(1), tensors(1)
    D.adamw_step(optimizer(want), 3)
    opt, side = optimizer(t), torch.cuda.Stream()
    torch.cuda.synchronize()
    held = busy(side)
    if call == "given":
        D.adamw_step(opt, 3, stream=side)
    else:
        with torch.cuda.stream(side):
            D.adamw_step(opt, 3)
    at, size = opt.table.data_ptr(), opt.table.numel()
    assert opt.away
    del opt
    again = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]  # (nothing is written to them)
    assert side.query() or all(a.data_ptr() != at for a in again)
    torch.cuda.synchronize()
    for n in t:
        assert torch.equal(t[n], want[n]), n
    del held


def test_an_optimizer_of_one_stream_goes_at_once():
    """On its own stream what comes next waits anyway: nothing to wait for on the host."""
    t = tensors(2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        opt = optimizer(t)
        side.synchronize()
        held = busy(side)
        D.adamw_step(opt, 1)
        assert not opt.away
        del opt
        assert not side.query()
    torch.cuda.synchronize()
    del held


def test_an_optimizer_that_goes_during_a_capture():
    """The capture stays whole, and the table waits for a later one."""
    a, b, want = tensors(3), tensors(4), tensors(4)
    D.adamw_step(optimizer(want), 1)
    side = torch.cuda.Stream()
    old, opt = optimizer(a), optimizer(b)
    D.adamw_step(old, 1, stream=side)
    torch.cuda.synchronize()
    at = old.table.data_ptr()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        D.adamw_step(opt, 1)
        del old
        gc.collect()
    assert [t.data_ptr() for t in D._left] == [at]
    graph.replay()
    torch.cuda.synchronize()
    for n in b:
        assert torch.equal(b[n], want[n]), n
    del graph, opt
    assert D._left == []
