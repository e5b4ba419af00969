"""The module that ops' small calls go through: what it leaves to the long way, without a GPU."""
import pytest
import torch

from structured_sparse_pretraining_b200 import _lib, ops

B = torch.bfloat16


@pytest.fixture(scope="module")
def calls():
    return ops._bind()


def test_what_is_no_cuda_tensor_is_left(calls):
    x, w, r = torch.zeros(2, 16, dtype=B), torch.zeros(16, dtype=B), torch.zeros(2)
    for first in (x, None, 3, "x", [x]):
        assert calls.rmsnorm(first, w, 1e-5, None, True, False, False, None, None, None, None, None) is None
        assert calls.rmsnorm_bwd(first, x, w, r, None, None, None) is None
        assert calls.quant_rows(first, None, None) is None
        assert calls.fwd_q8(first, r, x, r, x, None, None, 64, None) is None


def test_other_counts_of_arguments_are_left(calls):
    assert calls.rmsnorm() is None and calls.rmsnorm_bwd(None) is None
    assert calls.quant_rows(None) is None and calls.fwd_q8(*[None] * 10) is None


@pytest.mark.parametrize("args", [(), (1, 2, 3, 4), (0, 1, 1, 1, 1), ("a",) * 5])
def test_bind_refuses(calls, args):
    with pytest.raises((TypeError, ValueError)):
        calls.bind(*args)


def test_ops_refuse_with_the_long_ways_messages():
    with pytest.raises(ValueError, match="X"):
        ops.rmsnorm(torch.zeros(2, 16, dtype=B), torch.zeros(16, dtype=B), 1e-5)
    with pytest.raises(ValueError, match="A"):
        ops.quant_rows(torch.zeros(2, 16))


def test_status_raised():
    assert ops._done((1, 2)) == (1, 2)
    lib = _lib.load()
    rc = lib.slope_quant_rows(None, 1, 16, None, None, None)
    with pytest.raises(_lib.SlopeError) as e:
        ops._done(rc)
    assert e.value.code == rc == 1 and "NULL" in str(e.value)
