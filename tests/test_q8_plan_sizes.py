"""slope_q8_plan refuses the sizes that slope_fwd_q8 refuses, with the same status (host only)."""
import ctypes

import pytest

from structured_sparse_pretraining_b200 import _lib


@pytest.mark.parametrize("M,T,K,r", [(64, 0, 64, 0), (64, -4, 64, 0), (64, (1 << 30) + 1, 64, 0), (64, 1, 0, 0), (64, 1, 96, 0), (64, 1, -64, 0),
                                     (64, 1, 131136, 0), (100, 1, 64, 0), (0, 1, 64, 0), ((1 << 30) + 64, 1, 64, 0), (64, 1, 64, 12),
                                     (64, 1, 64, 264), (64, 1, 64, -8), (1 << 62, 1 << 40, 64, 0)])
def test_same_refusals(M, T, K, r):
    lib, raw = _lib.load(), (ctypes.c_uint8 * 4096)()
    b = (ctypes.addressof(raw) + 15) & ~15
    want = lib.slope_fwd_q8(b, b, b, b, b, b, b, T, K, M, r, b, None)
    x = ctypes.c_int(7)
    assert want in (1, 2)
    assert lib.slope_q8_plan(M, T, K, r, 148, ctypes.byref(x), ctypes.byref(x), ctypes.byref(x)) == want
    assert x.value == 7


@pytest.mark.parametrize("sms", [0, -1])
def test_no_sms(sms):
    x = ctypes.c_int(7)
    assert _lib.load().slope_q8_plan(64, 1, 64, 0, sms, ctypes.byref(x), ctypes.byref(x), ctypes.byref(x)) == 1
