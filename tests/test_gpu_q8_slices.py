"""Slices of a batch through the int8 path: scales and statistics that do not start on 16 bytes."""
import pytest
import torch

import q8_plain as P
from structured_sparse_pretraining_b200 import ops
from test_gpu_calls import LongWay

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(params=["short", "long"], autouse=True)
def way(request, monkeypatch):
    if request.param == "long":
        monkeypatch.setattr(ops, "_calls", LongWay())


@pytest.mark.parametrize("first", [1, 2, 3, 4])
@pytest.mark.parametrize("T,K,M,r", [(9, 512, 320, 16), (300, 1024, 1024, 0), (2000, 1024, 2560, 64)])
def test_fwd_q8_of_the_last_tokens(first, T, K, M, r):
    Xq, xs = ops.quant_rows(P.random_bf16((T, K), 1.0, 1))
    vq, ws = ops.quant_rows(P.random_bf16((M, K // 2), 0.02, 2))
    meta = P.random_codes(M, K, 3)
    XL, R = (P.random_bf16((T, r), 1.0, 4), P.random_bf16((r, M), 0.1, 5)) if r else (None, None)
    XLs = XL[first:] if r else None
    Y = ops.fwd_q8(Xq[first:], xs[first:], vq, ws, meta, XLs, R, M)
    aligned = ops.fwd_q8(Xq[first:], xs[first:].clone(), vq, ws, meta, XLs, R, M)
    assert torch.equal(Y, aligned)
    held = torch.empty(M + 1, device="cuda")
    held[1:] = ws
    assert torch.equal(ops.fwd_q8(Xq[first:], xs[first:], vq, held[1:], meta, XLs, R, M), aligned)


@pytest.mark.parametrize("T,D", [(9, 256), (1500, 1024)])
def test_outputs_into_slices(T, D):
    X, e, w = P.random_bf16((T, D), 1.0, 1), P.random_bf16((T, D), 2.0, 2), P.random_bf16((D,), 1.0, 3)
    want = ops.rmsnorm_q8(X, w, EPS, res=e, with_y=True, with_rstd=True)
    Q, s, rs = torch.zeros(T + 3, D, dtype=torch.int8, device="cuda"), torch.zeros(T + 3, device="cuda"), torch.zeros(T + 1, device="cuda")
    got = ops.rmsnorm_q8(X, w, EPS, res=e, with_y=True, Q=Q[3:], qscale=s[3:], rstd=rs[1:])
    assert got[1].data_ptr() == s[3:].data_ptr() and got[4].data_ptr() == rs[1:].data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not s[:3].any() and not rs[:1].any() and not Q[:3].any()
    Q2, s2 = ops.quant_rows(X, scale=s[1:T + 1])
    Q1, s1 = ops.quant_rows(X)
    assert torch.equal(Q1, Q2) and torch.equal(s1, s[1:T + 1]) and s[0] == 0
    dw = torch.zeros(D + 2, device="cuda")
    a = ops.rmsnorm_bwd(e, X, w, rs[1:], dw=dw[1:D + 1])
    b = ops.rmsnorm_bwd(e, X, w, want[4])
    assert torch.equal(a[0], b[0]) and torch.equal(dw[1:D + 1], b[1]) and dw[0] == 0 and dw[D + 1] == 0


def test_captured():
    X, w = P.random_bf16((9, 256), 1.0, 1), P.random_bf16((256,), 1.0, 2)
    s = torch.zeros(12, device="cuda")
    want = ops.quant_rows(X)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q, _ = ops.quant_rows(X, scale=s[3:])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Q, want[0]) and torch.equal(s[3:], want[1])


def test_overlaps_are_refused_there_too():
    X, e, w = P.random_bf16((9, 256), 1.0, 1), P.random_bf16((9, 256), 2.0, 2), P.random_bf16((256,), 1.0, 3)
    s = torch.zeros(40, device="cuda")
    with pytest.raises(ValueError, match="qscale overlaps rstd"):
        ops.rmsnorm_q8(X, w, EPS, qscale=s[1:10], rstd=s[5:14])
    with pytest.raises(ValueError, match="qscale overlaps rstd"):
        v = s[1:10]
        ops.rmsnorm_q8(X, w, EPS, qscale=v, rstd=v)
    with pytest.raises(ValueError, match="scale overlaps A"):
        ops.quant_rows(X, scale=X.view(torch.float32).view(-1)[1:10])
    rstd = torch.ones(400, device="cuda")
    with pytest.raises(ValueError, match="dw overlaps rstd"):
        ops.rmsnorm_bwd(e, X, w, rstd[1:10], dw=rstd[7:263])
    assert not s.any() and (rstd == 1).all()
    ops.rmsnorm_q8(X, w, EPS, qscale=s[1:10], rstd=s[10:19])
    assert s[1:19].all() and not s[0] and not s[19:].any()
