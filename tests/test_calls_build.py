"""The library without the module _calls, and when that is built again (no GPU)."""
import os
import subprocess
import sys
import types
import warnings

import pytest
import torch

from structured_sparse_pretraining_b200 import build, ops

B = torch.bfloat16


@pytest.fixture
def unbound(monkeypatch):
    monkeypatch.setattr(ops, "_calls", None)


def test_built_for_this_python_and_torch():
    assert build.calls_current()
    assert build.build_calls() == build.CALLS


def test_ops_work_without_it(unbound, monkeypatch):
    monkeypatch.setattr(build, "calls_key", lambda: "another torch")
    assert not build.calls_current()
    with pytest.warns(RuntimeWarning, match="_calls.so is not used"):
        with pytest.raises(ValueError, match="X must be a CUDA tensor"):
            ops.rmsnorm(torch.zeros(2, 16, dtype=B), torch.zeros(16, dtype=B), 1e-5)
    with warnings.catch_warnings():  # once
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="A must be a CUDA tensor"):
            ops.quant_rows(torch.zeros(2, 16, dtype=B))
        with pytest.raises(ValueError, match="CUDA"):
            ops.fwd_q8(torch.zeros(2, 64, dtype=torch.int8), None, None, None, None, None, None, 64)
        with pytest.raises(ValueError, match="CUDA"):
            ops.rmsnorm_bwd(torch.zeros(2, 16, dtype=B), None, None, None)


def test_ops_work_where_it_is_missing(unbound, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "none.so"))
    with pytest.warns(RuntimeWarning), pytest.raises(ValueError, match="A must be a CUDA tensor"):
        ops.quant_rows(torch.zeros(2, 16, dtype=B))


@pytest.mark.parametrize("how", ["fails", "missing"])
def test_the_library_builds_without_it(monkeypatch, capfd, how):
    real = subprocess.run

    def run(cmd, **kw):
        if cmd[0] != "g++":
            return real(cmd, **kw)
        if how == "missing":
            raise FileNotFoundError("g++")
        return types.SimpleNamespace(returncode=1, stdout="", stderr="no headers")
    monkeypatch.setattr(build, "calls_key", lambda: "another torch")  # so that it is built again
    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build(debug=False) == build.LIB and os.path.exists(build.LIB)
    assert build.build() == build.LIB
    assert "_calls.so not built" in capfd.readouterr().err


def test_another_torch_builds_it_again(monkeypatch):
    seen = []

    def run(cmd, **kw):
        seen.append(cmd)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build.subprocess, "run", run)
    build.build_calls()
    assert not seen
    monkeypatch.setattr(build, "calls_key", lambda: "another torch")
    build.build_calls()
    assert len(seen) == 1 and seen[0][0] == "g++" and '-DSLOPE_CALLS_KEY="another torch"' in seen[0]


def test_unbound_module_leaves_every_call():
    """Imported on its own, before ops has given it the entry points."""
    code = ("import torch; from structured_sparse_pretraining_b200 import _calls as c; b = torch.bfloat16\n"
            "dev = 'cuda' if torch.cuda.is_available() else 'cpu'\n"
            "x, w = torch.zeros(2, 16, dtype=b, device=dev), torch.zeros(16, dtype=b, device=dev)\n"
            "r = torch.zeros(2, device=dev)\n"
            "assert c.rmsnorm(x, w, 1e-5, None, True, False, False, None, None, None, None, None) is None\n"
            "assert c.rmsnorm_bwd(x, x, w, r, None, None, None) is None and c.quant_rows(x, None, None) is None\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


@pytest.mark.gpu
def test_results_are_the_same_without_it(unbound, monkeypatch):
    x, w = torch.randn(5, 256, device="cuda").to(B), torch.randn(256, device="cuda").to(B)
    want = ops.rmsnorm_q8(x, w, 1e-5, with_y=True)
    monkeypatch.setattr(ops, "_calls", None)
    monkeypatch.setattr(build, "calls_key", lambda: "another torch")
    with pytest.warns(RuntimeWarning):
        got = ops.rmsnorm_q8(x, w, 1e-5, with_y=True)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    assert ops._calls is ops._NoCalls


@pytest.mark.gpu
def test_unbound_module_leaves_cuda_tensors():
    test_unbound_module_leaves_every_call()
