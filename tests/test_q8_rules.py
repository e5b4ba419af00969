"""Host-only checks of the int8 path's calls: what they refuse before touching
the device, the scratch query, and the plain forms the GPU tests compare with."""
import ctypes

import pytest
import torch

import q8_plain as P
from structured_sparse_pretraining_b200 import _lib, ops


@pytest.fixture
def buf():
    raw = (ctypes.c_uint8 * 4096)()
    buf.keep = raw
    return (ctypes.addressof(raw) + 15) & ~15


def norm(lib, b, X=1, res=0, w=1, T=4, D=64, eps=1e-5, H=0, Y=1, Q=0, qscale=0, rstd=0):
    a = [b * v if v in (0, 1) else v for v in (X, res, w, H, Y, Q, qscale, rstd)]
    return lib.slope_rmsnorm(a[0] or None, a[1] or None, a[2] or None, T, D, eps, a[3] or None, a[4] or None, a[5] or None,
                             a[6] or None, a[7] or None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=0), 1), (dict(w=0), 1), (dict(Y=0), 1), (dict(Q=1), 1), (dict(H=1), 1), (dict(T=0), 1), (dict(T=-1), 1),
    (dict(T=1 << 31), 2), (dict(D=0), 1), (dict(D=-8), 1), (dict(D=12), 2), (dict(D=32776), 2), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1)])
def test_rmsnorm_refusals(buf, kw, code):
    assert norm(_lib.load(), buf, **kw) == code


@pytest.mark.parametrize("which", ["X", "res", "w", "H", "Y", "Q", "qscale", "rstd"])
def test_rmsnorm_alignment(buf, which):
    kw = dict(res=1, H=1, Q=1, qscale=1, rstd=1)
    kw[which] = buf + 8
    assert norm(_lib.load(), buf, **kw) == 3


def test_rmsnorm_bwd_refusals_and_scratch(buf):
    lib, b = _lib.load(), buf
    n = ctypes.c_int64(0)
    assert lib.slope_rmsnorm_bwd_ws(4, 64, None) == 1
    assert lib.slope_rmsnorm_bwd_ws(0, 64, ctypes.byref(n)) == 1
    assert lib.slope_rmsnorm_bwd_ws(4, 60, ctypes.byref(n)) == 2
    for T, D in ((1, 8), (4, 64), (1024, 5120), (8192, 32768)):
        assert lib.slope_rmsnorm_bwd_ws(T, D, ctypes.byref(n)) == 0 and n.value == 0
    for T, D in ((1025, 8), (8192, 5120), (1 << 30, 12288)):
        assert lib.slope_rmsnorm_bwd_ws(T, D, ctypes.byref(n)) == 0 and n.value >= D and n.value % D == 0

    far = b + (1 << 32)  # never read: every call here is refused

    def call(dY=b, H=b, w=b, rstd=b, dres=None, T=2000, D=64, dH=far, dw=b, ws=b, floats=1 << 20):
        return lib.slope_rmsnorm_bwd(dY, H, w, rstd, dres, T, D, dH, dw, ws, floats, None)
    assert lib.slope_rmsnorm_bwd_ws(2000, 64, ctypes.byref(n)) == 0
    assert call(floats=n.value - 1) == 2
    for name in ("dY", "H", "w", "rstd", "dH", "dw", "ws"):
        assert call(**{name: None}) == 1
        assert call(**{name: b + 4}) == 3
    assert call(dres=b + 8) == 3
    assert call(T=0) == 1
    assert call(D=20) == 2
    for T in (4, 2000):  # dH over dY or H, wholly or by its last row
        assert call(T=T, dH=b) == 1
        assert call(T=T, H=far, dH=far) == 1
        assert call(T=T, dH=b + 128 * (T - 1)) == 1
        assert call(T=T, dY=far + 128 * (T - 1)) == 1
        assert call(T=T, dres=far + 128) == 1


@pytest.mark.parametrize("rows,K,code", [(0, 64, 1), (4, 0, 1), (4, 20, 2), (4, 65544, 2), ((1 << 30) + 1, 8, 2)])
def test_quant_rows_refusals(buf, rows, K, code):
    lib = _lib.load()
    assert lib.slope_quant_rows(buf, rows, K, buf, buf, None) == code
    assert lib.slope_quant_rows(None, 4, 64, buf, buf, None) == 1
    assert lib.slope_quant_rows(buf, 4, 64, buf + 4, buf, None) == 3


@pytest.mark.parametrize("T,K,M,r,code", [(0, 64, 64, 0, 1), (4, 96, 64, 0, 2), (4, 64, 100, 0, 2), (4, 131136, 64, 0, 2),
                                          (4, 64, 64, 12, 2), (4, 64, 64, 264, 2), (4, 64, 64, -8, 1), (4, -64, 64, 0, 1)])
def test_fwd_q8_refusals(buf, T, K, M, r, code):
    b = buf
    assert _lib.load().slope_fwd_q8(b, b, b, b, b, b, b, T, K, M, r, b, None) == code


def test_fwd_q8_pointers(buf):
    lib, b = _lib.load(), buf
    for i in (0, 1, 2, 3, 4, 5, 6):
        a = [b] * 7
        a[i] = None
        assert lib.slope_fwd_q8(*a, 4, 64, 64, 8, b, None) == 1
        a[i] = b + 8
        assert lib.slope_fwd_q8(*a, 4, 64, 64, 8, b, None) == 3
    assert lib.slope_fwd_q8(b, b, b, b, b, None, None, 4, 64, 64, 0, None, None) == 1


def test_ops_refuse_cpu_tensors_and_wrong_types():
    X, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.rmsnorm(X, w, 1e-5)
    with pytest.raises(ValueError, match="CUDA"):
        ops.quant_rows(X)
    with pytest.raises(ValueError, match="CUDA"):
        ops.fwd_q8(X.to(torch.int8), w, X, w, X, None, None, 64)


@pytest.mark.parametrize("M,T,K,r", [(64, 1, 64, 0), (64, 5000, 4096, 8), (128, 1, 64, 0), (192, 300, 131072, 256), (27648, 1, 9216, 96),
                                     (9216, 16, 36864, 96), (36864, 8192, 9216, 96), (1024, 333, 4096, 0), (512, 16, 16384, 64)])
def test_q8_plan_is_well_formed(M, T, K, r):
    rows, bn, splits = ops.q8_plan(M, T, K, r)
    kts = -(-K // 256)
    if rows == 0:
        assert T <= 4 and bn in (1, 2, 4) and splits in (1, 2, 4, 8, 16)
        assert bn * -(-K // 1024) * 1024 <= 200 * 1024, "the tokens' rows fit shared memory"
    elif rows == 128:
        assert bn in (16, 32, 64, 128) and splits in (1, 2, 3, 4, 8) and splits <= kts
    else:
        assert (rows, bn) in ((256, 256), (512, 224)) and M >= 128 and splits == 1


def test_q8_plan_of_the_largest_layers():
    """Weight streaming on clusters at a decode step, 256-row tiles at a few hundred tokens, 512-row ones at a prefill batch, CUDA cores for one token
    of a small layer."""
    assert ops.q8_plan(27648, 1, 9216, 96) == (128, 16, 2)
    assert ops.q8_plan(9216, 16, 36864, 96) == (128, 16, 2)
    assert ops.q8_plan(36864, 8192, 9216, 96) == (512, 224, 1)
    assert ops.q8_plan(27648, 256, 9216, 96) == (256, 256, 1)
    assert ops.q8_plan(1024, 1, 1024, 64)[0] == 0
    lib = _lib.load()
    assert lib.slope_q8_plan(64, 1, 64, 0, 148, None, None, None) == 1
    x = ctypes.c_int(0)
    assert lib.slope_q8_plan(0, 1, 64, 0, 148, ctypes.byref(x), ctypes.byref(x), ctypes.byref(x)) == 1


# ------------------------------------------------------------------ the plain forms themselves
def test_plain_norm_gradient_is_the_forward_s_derivative():
    """norm_bwd against autograd of the forward formula and against central differences, in 64 bits."""
    g = torch.Generator().manual_seed(3)
    T, D, eps = 5, 24, 1e-3
    h = torch.randn(T, D, generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(D, generator=g, dtype=torch.float64)
    dY = torch.randn(T, D, generator=g, dtype=torch.float64)

    def fwd(h, w):
        return ((h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * w) * dY).sum()
    rstd = (h.square().mean(1) + eps).rsqrt()
    dh, dw, _, _ = P.norm_bwd(dY, h, w, rstd)
    ha, wa = h.clone().requires_grad_(), w.clone().requires_grad_()
    fwd(ha, wa).backward()
    assert torch.allclose(dh, ha.grad, rtol=1e-12, atol=1e-13) and torch.allclose(dw, wa.grad, rtol=1e-12, atol=1e-13)
    step = 1e-6
    for t, d in ((0, 0), (2, 7), (4, 23)):
        e = torch.zeros_like(h)
        e[t, d] = step
        assert abs((fwd(h + e, w) - fwd(h - e, w)) / (2 * step) - dh[t, d]) < 1e-8
        assert abs((fwd(h, w + e[t]) - fwd(h, w - e[t])) / (2 * step) - dw[d]) < 1e-8


def test_plain_dense_matches_the_oracle():
    import numpy as np

    import oracle
    from structured_sparse_pretraining_b200 import inputs as I
    W = I.normal_bf16((32, 128), 0.02, 3, 0, "W")
    vals, meta, _ = oracle.prune24(I.bits(W))
    v = I.from_bits(vals)
    m = torch.from_numpy(meta.view(np.int16).copy())
    want = I.from_bits(oracle.decompress(vals, meta, 128)).double()
    assert torch.equal(P.dense(v, m, 128), want)


def test_plain_quantise_rounds_ties_to_even():
    p = torch.tensor([[254.0, 1.0, 3.0, -1.0, -3.0, 5.0, 253.0, 0.0]], dtype=torch.float64)
    q, top = P.quantise(p)
    assert q.tolist() == [[127, 0, 2, 0, -2, 2, 126, 0]] and top.item() == 254.0
