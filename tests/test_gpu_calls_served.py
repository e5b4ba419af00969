"""That the int8 path's calls are served by the module _calls where everything
fits: what it leaves goes the long way and gives the same results, so the other
tests of these calls would pass without it."""
import pytest
import torch

from structured_sparse_pretraining_b200 import ops
from test_gpu_calls import NAMES, LongWay, as_tuple, cases, tensors

pytestmark = pytest.mark.gpu


class Recorder:
    """Stands for _calls: passes each call on and notes the function's name and whether it was served."""
    def __init__(self, calls):
        self.calls, self.seen = calls, []

    def __getattr__(self, name):
        def run(*a):
            out = getattr(self.calls, name)(*a)
            self.seen.append((name, out is not None))
            return out
        return run


FUNCTION = {n: "rmsnorm" if n.startswith("norm") else "rmsnorm_bwd" if n.startswith("bwd") else "quant_rows" if n == "quant" else "fwd_q8"
            for n in NAMES}


@pytest.mark.parametrize("name", NAMES)
def test_each_call_is_served(name, monkeypatch):
    f = cases(tensors())[name]
    f()
    r = Recorder(ops._bind())
    monkeypatch.setattr(ops, "_calls", r)
    out = as_tuple(f())
    assert r.seen == [(FUNCTION[name], True)]
    # and with every output given
    t = tensors()
    xq, xs = ops.quant_rows(t["X"])
    wq, ws = ops.quant_rows(t["W"])
    del r.seen[:]
    if name == "norm":
        ops.rmsnorm(t["X"], t["w"], 1e-5, Y=out[0])
    elif name == "norm_q8_all":
        ops.rmsnorm_q8(t["X"], t["w"], 1e-5, res=t["res"], Q=out[0], qscale=out[1], Y=out[2], H=out[3], rstd=out[4])
    elif name == "bwd_res":
        ops.rmsnorm_bwd(t["dY"], t["X"], t["w"], t["rstd"], dres=t["res"], dH=out[0], dw=out[1])
    elif name == "quant":
        ops.quant_rows(t["X"], Q=out[0], scale=out[1])
    elif name == "q8_adapter":
        ops.fwd_q8(xq, xs, wq, ws, t["meta"], t["XL"], t["Rm"], t["meta"].shape[0], Y=out[0])
    assert all(served for _, served in r.seen)


@pytest.mark.parametrize("name", NAMES)
def test_the_long_way_does_not_touch_it(name, monkeypatch):
    f = cases(tensors())[name]
    r = Recorder(ops._bind())
    monkeypatch.setattr(ops, "_calls", LongWay())
    f()
    assert r.seen == []


def test_gradients_with_scratch_are_served(monkeypatch):
    x, w = torch.randn(1500, 64, device="cuda").to(torch.bfloat16), torch.ones(64, device="cuda", dtype=torch.bfloat16)
    r = Recorder(ops._bind())
    monkeypatch.setattr(ops, "_calls", r)
    ops.rmsnorm_bwd(x, x, w, torch.rand(1500, device="cuda"))
    assert r.seen == [("rmsnorm_bwd", True)]


def test_parameters_on_another_stream_and_in_a_graph_are_served(monkeypatch):
    t = tensors()
    w = torch.nn.Parameter(t["w"].clone())
    r = Recorder(ops._bind())
    monkeypatch.setattr(ops, "_calls", r)
    ops.rmsnorm(t["X"], w, 1e-5)
    with torch.cuda.stream(torch.cuda.Stream()):
        ops.rmsnorm(t["X"], t["w"], 1e-5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.rmsnorm(t["X"], t["w"], 1e-5)
    torch.cuda.synchronize()
    assert r.seen == [("rmsnorm", True)] * 3
