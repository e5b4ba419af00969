"""The int8 path's calls through the module _calls against the same calls the
long way (which the module leaves what does not fit): the same bits, the same
errors, and no reference or memory kept."""
import gc
import sys
import threading

import pytest
import torch

from structured_sparse_pretraining_b200 import _lib, ops

pytestmark = pytest.mark.gpu
B = torch.bfloat16
T, D, N, R = 5, 256, 128, 16


class LongWay:
    """Stands for _calls: everything is left to the long way."""
    def __getattr__(self, name):
        return lambda *a: None


@pytest.fixture
def long_way(monkeypatch):
    def run(f):
        with monkeypatch.context() as m:
            m.setattr(ops, "_calls", LongWay())
            return f()
    return run


def tensors(seed=0, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g).to(B).to(dev)  # noqa: E731
    t = dict(X=rand(T, D), res=rand(T, D), w=rand(D), dY=rand(T, D), W=rand(N, D // 2), XL=rand(T, R), Rm=rand(R, N))
    t["rstd"] = torch.rand(T, generator=g).to(dev)
    t["meta"] = torch.full((N, D // 16), 0x4444, dtype=torch.int16, device=dev)
    return t


def cases(t):
    X, w = t["X"], t["w"]
    xq, xs = ops.quant_rows(X)
    wq, ws = ops.quant_rows(t["W"])
    return {
        "norm": lambda: ops.rmsnorm(X, w, 1e-5),
        "norm_res_rstd": lambda: ops.rmsnorm(X, w, 1e-5, res=t["res"], with_rstd=True),
        "norm_q8": lambda: ops.rmsnorm_q8(X, w, 1e-5),
        "norm_q8_all": lambda: ops.rmsnorm_q8(X, w, 1e-5, res=t["res"], with_y=True, with_rstd=True),
        "bwd": lambda: ops.rmsnorm_bwd(t["dY"], X, w, t["rstd"]),
        "bwd_res": lambda: ops.rmsnorm_bwd(t["dY"], X, w, t["rstd"], dres=t["res"]),
        "quant": lambda: ops.quant_rows(X),
        "q8": lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], None, None, N),
        "q8_adapter": lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], t["XL"], t["Rm"], N),
    }


def as_tuple(v):
    return v if isinstance(v, tuple) else (v,)


NAMES = ["norm", "norm_res_rstd", "norm_q8", "norm_q8_all", "bwd", "bwd_res", "quant", "q8", "q8_adapter"]


@pytest.mark.parametrize("name", NAMES)
def test_same_as_the_long_way(name, long_way):
    f = cases(tensors())[name]
    a, b = as_tuple(f()), as_tuple(long_way(f))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and x.device == y.device
            assert not x.requires_grad and torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_rows_for_two_launches_of_the_gradients(long_way):
    x, w = torch.randn(1500, 64, device="cuda").to(B), torch.ones(64, device="cuda", dtype=B)
    r = torch.rand(1500, device="cuda")
    a, b = ops.rmsnorm_bwd(x, x, w, r), long_way(lambda: ops.rmsnorm_bwd(x, x, w, r))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_given_outputs_are_returned():
    t = tensors()
    X, w = t["X"], t["w"]
    Q, s = torch.empty(T, D, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    H, Y, r = torch.empty_like(X), torch.empty_like(X), torch.empty(T, device="cuda")
    out = ops.rmsnorm_q8(X, w, 1e-5, res=t["res"], H=H, Y=Y, Q=Q, qscale=s, rstd=r)
    assert all(a is b for a, b in zip(out, (Q, s, Y, H, r)))
    out = ops.rmsnorm(X, w, 1e-5, res=t["res"], H=H, Y=Y, rstd=r)
    assert all(a is b for a, b in zip(out, (Y, H, r)))
    assert all(a is b for a, b in zip(ops.quant_rows(X, Q, s), (Q, s)))
    dw = torch.empty(D, device="cuda")
    assert all(a is b for a, b in zip(ops.rmsnorm_bwd(t["dY"], X, w, r, dH=H, dw=dw), (H, dw)))
    wq, ws = ops.quant_rows(t["W"])
    y = torch.empty(T, N, dtype=B, device="cuda")
    assert ops.fwd_q8(Q, s, wq, ws, t["meta"], None, None, N, Y=y) is y


@pytest.mark.parametrize("name", NAMES)
def test_no_reference_and_no_memory_kept(name):
    t = tensors()
    f = cases(t)[name]
    out = as_tuple(f())
    assert all(o is None or sys.getrefcount(o) == 3 for o in out)  # the tuple, the loop's name and the argument
    del out
    gc.collect()
    counts, held = {k: sys.getrefcount(v) for k, v in t.items()}, torch.cuda.memory_allocated()
    for _ in range(200):
        f()
    assert torch.cuda.memory_allocated() == held
    assert counts == {k: sys.getrefcount(v) for k, v in t.items()}


def test_what_does_not_fit_is_refused_as_before(long_way):
    t = tensors()
    X, w, rstd = t["X"], t["w"], t["rstd"]
    xq, xs = ops.quant_rows(X)
    wq, ws = ops.quant_rows(t["W"])
    calls = [
        lambda: ops.rmsnorm(X, w[:-8], 1e-5),
        lambda: ops.rmsnorm(X, w.float(), 1e-5),
        lambda: ops.rmsnorm(X[:, ::2], w[::2], 1e-5),
        lambda: ops.rmsnorm(X, w, -1.0),
        lambda: ops.rmsnorm(X, w, float("nan")),
        lambda: ops.rmsnorm(X, w, 1e-5, H=X),
        lambda: ops.rmsnorm(X, w, 1e-5, Y=X[:3]),
        lambda: ops.rmsnorm(X.cpu(), w, 1e-5),
        lambda: ops.rmsnorm(X, w.cpu(), 1e-5),
        lambda: ops.rmsnorm(X[:, :252].contiguous(), w[:252].contiguous(), 1e-5),
        lambda: ops.rmsnorm(X[:0], w, 1e-5),
        lambda: ops.rmsnorm(X[0], w, 1e-5),
        lambda: ops.rmsnorm_bwd(X, X, w, rstd[:-1]),
        lambda: ops.rmsnorm_bwd(X, X, w, rstd, dw=w),
        lambda: ops.rmsnorm_bwd(X[:0], X[:0], w, rstd[:0]),
        lambda: ops.quant_rows(X, Q=X),
        lambda: ops.quant_rows(X.float()),
        lambda: ops.quant_rows(X[:, :12].contiguous()),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], t["XL"], None, N),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], None, t["Rm"], N),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], t["XL"], t["Rm"][:, :64], N),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"].int(), None, None, N),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], None, None, 64),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], None, None, -64),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], None, None, 2 ** 70),
        lambda: ops.fwd_q8(xq, xs, wq[:, :126].contiguous(), ws, t["meta"], None, None, N),
        lambda: ops.fwd_q8(xq, xs, wq, ws, t["meta"], t["XL"][:, :4].contiguous(), t["Rm"][:4].contiguous(), N),
    ]
    for i, f in enumerate(calls):
        seen = []
        for run in (lambda g: g(), long_way):
            with pytest.raises((ValueError, TypeError, _lib.SlopeError, OverflowError, AttributeError)) as e:
                run(f)
            seen.append((type(e.value), str(e.value)))
        assert seen[0] == seen[1], (i, seen)


def test_parameters_and_subclasses():
    t = tensors()
    w = torch.nn.Parameter(t["w"].clone())

    class Sub(torch.Tensor):
        pass

    want = ops.rmsnorm(t["X"], t["w"], 1e-5)[0]
    assert torch.equal(ops.rmsnorm(t["X"], w, 1e-5)[0], want)
    assert torch.equal(ops.rmsnorm(t["X"].as_subclass(Sub), w, 1e-5)[0], want)


def test_on_another_stream_and_in_a_graph():
    t = tensors()
    fs = cases(t)
    want = {k: as_tuple(f()) for k, f in fs.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        side = {k: as_tuple(f()) for k, f in fs.items()}
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = {k: as_tuple(f()) for k, f in fs.items()}
    g.replay()
    torch.cuda.synchronize()
    for got in (side, held):
        for k in fs:
            for a, b in zip(got[k], want[k]):
                assert (a is None and b is None) or torch.equal(a, b), k


def test_two_threads_at_once():
    t = [tensors(i) for i in range(2)]
    want = [{k: as_tuple(f()) for k, f in cases(u).items()} for u in t]
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            fs = cases(t[i])
            for _ in range(50):
                for k, f in fs.items():
                    for a, b in zip(as_tuple(f()), want[i][k]):
                        if a is not None and not torch.equal(a, b):
                            bad.append((i, k))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [th.start() for th in threads]
    [th.join() for th in threads]
    assert not bad
