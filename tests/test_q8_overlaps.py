"""What the int8 path's calls refuse among overlapping buffers, before touching the device."""
import ctypes

import pytest

from structured_sparse_pretraining_b200 import _lib

ARG = 1
STEP = 1 << 24  # apart: further than any buffer here is long; nothing at these addresses is read


def at(i):
    return (i + 1) * STEP


@pytest.fixture
def lib():
    return _lib.load()


def refused(lib, rc, *names):
    """SLOPE_ERR_ARG with both buffers named; None where the overlap was accepted (the call then stops for want of a device)."""
    if rc == ARG:
        msg = lib.slope_last_error().decode()
        assert "overlaps" in msg and all(n in msg for n in names), msg
        return True
    assert rc in (6, 7), rc  # no device in this process
    return False


T, D = 40, 64
NORM = ["X", "res", "w", "H", "Y", "Q", "qscale", "rstd"]
NORM_BYTES = dict(X=2 * T * D, res=2 * T * D, w=2 * D, H=2 * T * D, Y=2 * T * D, Q=T * D, qscale=4 * T, rstd=4 * T)


def norm(lib, **where):
    p = {n: where.get(n, at(i)) for i, n in enumerate(NORM)}
    return lib.slope_rmsnorm(p["X"], p["res"], p["w"], T, D, 1e-5, p["H"], p["Y"], p["Q"], p["qscale"], p["rstd"], None)


@pytest.fixture(autouse=True)
def _no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the accepted calls here have addresses that only a process without a device may pass")


@pytest.mark.parametrize("out", NORM[3:])
@pytest.mark.parametrize("other", NORM)
def test_rmsnorm(lib, out, other):
    if out == other:
        return
    i = at(NORM.index(other))
    whole = refused(lib, norm(lib, **{out: i}), out, other)
    assert whole == (not (out in ("H", "Y") and other in ("X", "res")))
    inner = i + NORM_BYTES[other] - 16  # the last bytes of the other
    assert refused(lib, norm(lib, **{out: inner}), out, other)
    assert not refused(lib, norm(lib, **{out: i + NORM_BYTES[other]}))
    if NORM_BYTES[out] > 16:
        assert refused(lib, norm(lib, **{out: i - NORM_BYTES[out] + 16}), out, other)
    assert not refused(lib, norm(lib, **{out: i - NORM_BYTES[out]}))


def test_rmsnorm_in_place_is_taken(lib):
    x, e = at(0), at(1)
    for kw in (dict(), dict(H=x, Y=e), dict(H=e, Y=x), dict(H=e), dict(Y=x), dict(res=x), dict(res=x, H=x)):
        assert not refused(lib, norm(lib, **kw))
    assert refused(lib, norm(lib, H=x, Y=x), "H", "Y")


def test_quant_rows(lib):
    rows, K = 40, 64
    names, size = ["A", "Q", "scale"], dict(A=2 * rows * K, Q=rows * K, scale=4 * rows)

    def call(**where):
        p = {n: where.get(n, at(i)) for i, n in enumerate(names)}
        return lib.slope_quant_rows(p["A"], rows, K, p["Q"], p["scale"], None)
    assert not refused(lib, call())
    for out in ("Q", "scale"):
        for other in names:
            if other != out:
                i = at(names.index(other))
                for place in (i, i + size[other] - 16, i - size[out] + 16):
                    assert refused(lib, call(**{out: place}), out, other)
                for place in (i + size[other], i - size[out]):
                    assert not refused(lib, call(**{out: place}))


@pytest.mark.parametrize("rows", [40, 2000])
def test_rmsnorm_bwd(lib, rows):
    n = ctypes.c_int64(0)
    assert lib.slope_rmsnorm_bwd_ws(rows, D, ctypes.byref(n)) == 0
    names = ["dY", "H", "w", "rstd", "dres", "dH", "dw", "ws"]
    size = dict(dY=2 * rows * D, H=2 * rows * D, w=2 * D, rstd=4 * rows, dres=2 * rows * D, dH=2 * rows * D, dw=4 * D, ws=4 * n.value)

    def call(**where):
        p = {m: where.get(m, at(i)) for i, m in enumerate(names)}
        return lib.slope_rmsnorm_bwd(p["dY"], p["H"], p["w"], p["rstd"], p["dres"], rows, D, p["dH"], p["dw"], p["ws"], n.value, None)
    assert not refused(lib, call())
    assert not refused(lib, call(dH=at(names.index("dres"))))
    for out in ("dH", "dw") + (("ws",) if n.value else ()):
        for other in names:
            if other == out or not size[other]:
                continue
            i = at(names.index(other))
            for place in (i, i + size[other] - 16, i - size[out] + 16):
                if not (out == "dH" and other == "dres" and place == i):
                    assert call(**{out: place}) == ARG and "overlaps" in lib.slope_last_error().decode()
            assert not refused(lib, call(**{out: i + size[other]}))


def test_fwd_q8(lib):
    t, K, M, r = 40, 128, 64, 8
    names = ["Xq", "xscale", "vals_q", "wscale", "meta", "XL", "R", "Y"]
    size = dict(Xq=t * K, xscale=4 * t, vals_q=M * K // 2, wscale=4 * M, meta=M * K // 8, XL=2 * t * r, R=2 * r * M, Y=2 * t * M)

    def call(rank=r, **where):
        p = {n: where.get(n, at(i)) for i, n in enumerate(names)}
        return lib.slope_fwd_q8(p["Xq"], p["xscale"], p["vals_q"], p["wscale"], p["meta"], p["XL"], p["R"], t, K, M, rank, p["Y"], None)
    assert not refused(lib, call())
    for other in names[:-1]:
        i = at(names.index(other))
        for place in (i, i + size[other] - 16, i - size["Y"] + 16):
            assert refused(lib, call(Y=place), "Y", other)
    assert not refused(lib, call(rank=0, Y=at(names.index("R"))))
