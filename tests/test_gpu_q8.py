"""GPU tests of the int8 inference path (norm, its gradients, row quantiser, int8
sparse product) against plain 64-bit forms.  Integers must match exactly; the
tolerances of the rest are derived from the roundings each operator makes."""
import pytest
import torch

import q8_plain as P
from parity_util import _CANARY, check_guards, guarded_empty
from structured_sparse_pretraining_b200 import ops

pytestmark = pytest.mark.gpu
EPS = 1e-5
_CANARY.setdefault(torch.bfloat16, 0x7FA5)


@pytest.fixture(scope="module", autouse=True)
def _setup():
    ops.device_check()
    yield
    ops.status_sync()


def within(got, want, tol, what):
    """|got - want| <= tol everywhere, NaN where NaN is wanted."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    err = torch.where(nan | (got == want), 0.0, (got - want).abs() - tol)
    assert not (err > 0).any(), f"{what}: {float(err.max()):.3e} beyond the tolerance at {int(err.argmax())}"


def depth(D):
    """Longest chain of additions of a row sum: a thread's values (up to 64) and two five-step trees."""
    return 64 + 10


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("rows,K", [(1, 8), (3, 16), (5, 64), (130, 264), (33, 512), (7, 520), (4, 1000), (9, 1024), (6, 1032),
                                    (3, 4608), (2, 16384), (2, 16392), (2, 36864), (1, 65536), (2000, 96),
                                    (10000, 72), (9600, 512), (7201, 1000), (1000, 1032), (2049, 4608), (900, 8200), (700, 12288), (333, 36864), (300, 65536),
                                    (800, 12296), (700, 16384), (600, 18432), (500, 18440)])
def test_quant_rows(rows, K):
    A = P.random_bf16((rows, K), 0.02, 1)
    if rows > 2:
        A[1] = 0
    Q, scale = ops.quant_rows(A)
    q, top = P.quantise(A.double())
    assert torch.equal(Q, q)
    within(scale, top / 127, P.F32 * top / 127, "scale")  # one division


def test_quant_rows_decides_ties_and_borders_exactly():
    """Every quotient k + 1/2, just beside it, and every pair of bf16 significands at the border."""
    rows = []
    for top in (254.0, 127.0, 255.0 * 2 ** -20, 129.0 * 2 ** 30, 2.0 ** -126 * 254, 3.0e38, 1e-38, 9.2e-41 * 8):
        t = torch.tensor(top).to(torch.bfloat16).double()
        k = torch.arange(-127, 127, dtype=torch.float64)
        near = (t * (k + 0.5) / 127).to(torch.bfloat16)
        bits = near.view(torch.int16)
        v = torch.cat([(bits + d).view(torch.bfloat16) for d in (-1, 0, 1)])
        v = torch.where(v.double().abs() <= t, v, torch.zeros_like(v))
        rows.append(torch.cat([v, t.to(torch.bfloat16).view(1), torch.zeros(5, dtype=torch.bfloat16)]))
    A = torch.stack(rows).contiguous().cuda()
    assert A.shape[1] % 8 == 0
    Q, scale = ops.quant_rows(A)
    q, top = P.quantise(A.double())
    assert torch.equal(Q, q)
    within(scale, top / 127, P.F32 * top / 127 + 2.0 ** -149, "scale")  # the last place of a subnormal is 2^-149


def test_quant_rows_not_finite():
    A = P.random_bf16((6, 256), 1.0, 2)
    A[0, 3] = float("inf")
    A[2, 255] = float("-inf")
    A[3, 0] = float("nan")
    A[5] = 0
    Q, scale = ops.quant_rows(A)
    q, top = P.quantise(A.double())
    assert torch.equal(Q, q) and not Q[[0, 2, 3, 5]].any()
    assert torch.isnan(scale[[0, 2, 3]]).all() and scale[5] == 0
    within(scale, top / 127, P.F32 * torch.nan_to_num(top) / 127, "scale")


# ------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 8), (1, 9216), (5, 64), (7, 248), (9, 256), (6, 264), (3, 520), (130, 768), (4, 1000), (5, 1024), (3, 1032),
               (11, 5120), (2, 16384), (3, 16392), (2, 32768), (1027, 512),
              # many rows: the ring of rows, every number of chunks per thread, one and several stages' turns
              (5000, 64), (4801, 264), (7200, 520), (8000, 1000), (9001, 1024), (1100, 1040), (1201, 3080), (1333, 5120), (903, 6152), (950, 9216), (700, 12288), (400, 12296), (310, 24576), (300, 32768)]


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm(T, D, res):
    X, w = P.random_bf16((T, D), 1.0, 3), (1 + P.random_bf16((D,), 0.2, 4).float()).to(torch.bfloat16)
    e = P.random_bf16((T, D), 2.0, 5) if res else None
    if T > 3:
        X[2] = 0
        if res:
            e[2] = 0
    h, y, rstd, q, qs = P.norm(X, w, EPS, e)
    Y, H, rs = ops.rmsnorm(X, w, EPS, res=e, with_rstd=True)
    Q, s, Y8, H8, rs8 = ops.rmsnorm_q8(X, w, EPS, res=e, with_y=True, with_rstd=True)
    Q1, s1, none, _, none2 = ops.rmsnorm_q8(X, w, EPS, res=e)
    assert none is None and none2 is None and (H is None) == (not res)
    # rstd: the sum's depth and half of it through the root, then division, addition, root, reciprocal
    rel = (depth(D) / 2 + 4) * P.F32
    within(rs, rstd, rel * rstd, "rstd")
    within(Y, y, (P.BF16 * (1 + 2 * rel) + 2 * rel) * y.abs() + 2.0 ** -134, "Y")
    assert torch.equal(Q, q)
    within(s, qs, (rel + 3 * P.F32) * qs, "qscale")
    if res:
        assert torch.equal(H, h) and torch.equal(H8, h)
    for a, b in ((Y, Y8), (rs, rs8), (Q, Q1), (s, s1)):
        assert torch.equal(a, b)


def test_rmsnorm_q8_is_decided_by_h_and_w_alone():
    """Products of bf16 numbers right at the quantiser's borders: all 2^14 pairs of significands against one largest product."""
    sig = torch.arange(128, 256, dtype=torch.float32)
    h = sig.repeat_interleave(128) / 256
    w = sig.repeat(128) / 128
    for top in (255.0, 201.0, 129.0):
        for sign in (1, -1):
            X = torch.cat([sign * h, torch.tensor([top]), torch.zeros(7)]).to(torch.bfloat16).view(1, -1).cuda()
            wt = torch.cat([w, torch.ones(8)]).to(torch.bfloat16).cuda()
            X = torch.cat([X, X * 2.0 ** -7, X * 2.0 ** 60, X * 2.0 ** -90]).contiguous()
            X[1, -8] = top / 64
            Q, _, _, _, _ = ops.rmsnorm_q8(X, wt, EPS)
            q, _ = P.quantise(X.double() * wt.double())
            assert torch.equal(Q, q)


def test_rmsnorm_not_finite_and_huge():
    T, D = 6, 320
    X, w = P.random_bf16((T, D), 1.0, 6), torch.ones(D, dtype=torch.bfloat16, device="cuda")
    X[0, 5] = float("inf")
    X[1, 6] = float("nan")
    X[2] *= 2.0 ** 100  # squares overflow binary32
    X[3] = 0
    X[4] *= 2.0 ** -100
    Q, s, Y, _, rs = ops.rmsnorm_q8(X, w, EPS, with_y=True, with_rstd=True)
    h, y, rstd, q, qs = P.norm(X, w, EPS)
    assert torch.equal(Q, q)
    assert torch.isnan(s[:2]).all() and s[3] == 0
    rel = (depth(D) / 2 + 6) * P.F32
    within(rs[2:], rstd[2:], rel * rstd[2:], "rstd")
    within(s[2:], qs[2:], (rel + 3 * P.F32) * qs[2:], "qscale")
    within(Y[2:], y[2:], (P.BF16 + 3 * rel) * y[2:].abs() + 2.0 ** -134, "Y")
    assert rs[0] == 0 and torch.isnan(rs[1])
    assert torch.isnan(Y[0, 5]) and (Y[0, :5] == 0).all() and torch.isnan(Y[1]).all()
    # the same rows among many, wide: the ring's path through the same branches
    Xs = P.random_bf16((1200, 2560), 1.0, 6)
    Xs[3::7] *= 2.0 ** 100
    Xs[4::7, 9] = float("inf")
    Xs[5::7] = 0
    Xs[6::7, 2559] = float("nan")
    wq = torch.ones(2560, dtype=torch.bfloat16, device="cuda")
    Qs, ss, Ys, _, rss = ops.rmsnorm_q8(Xs, wq, EPS, with_y=True, with_rstd=True)
    _, ys, rstds, qs_, qss = P.norm(Xs, wq, EPS)
    assert torch.equal(Qs, qs_) and torch.isnan(ss[4::7]).all() and torch.isnan(ss[6::7]).all() and (rss[4::7] == 0).all()
    ok = torch.ones(1200, dtype=torch.bool)
    ok[4::7] = ok[6::7] = False
    within(rss[ok], rstds[ok], rel * rstds[ok], "rstd")
    within(ss[ok], qss[ok], (rel + 3 * P.F32) * qss[ok], "qscale")
    within(Ys[ok], ys[ok], (P.BF16 + 3 * rel) * ys[ok].abs() + 2.0 ** -134, "Y")
    Xs = Xs[:, :512].repeat(8, 1).contiguous()  # and by warps
    Qs, ss, Ys, _, rss = ops.rmsnorm_q8(Xs, wq[:512].contiguous(), EPS, with_y=True, with_rstd=True)
    _, ys, rstds, qs_, qss = P.norm(Xs, wq[:512], EPS)
    assert torch.equal(Qs, qs_) and torch.equal(torch.isnan(ss), torch.isnan(qss))
    ok = torch.isfinite(Xs.float()).all(1)
    within(rss[ok], rstds[ok], rel * rstds[ok], "rstd")
    within(ss[ok], qss[ok], (rel + 3 * P.F32) * qss[ok], "qscale")
    within(Ys[ok], ys[ok], (P.BF16 + 3 * rel) * ys[ok].abs() + 2.0 ** -134, "Y")
    # a wide row takes the CTA's path through the same branch
    Xw = P.random_bf16((2, 5120), 1.0, 7) * 2.0 ** 110
    Yw, _, rw = ops.rmsnorm(Xw, torch.ones(5120, dtype=torch.bfloat16, device="cuda"), EPS, with_rstd=True)
    _, yw, rstdw, _, _ = P.norm(Xw, torch.ones(5120, dtype=torch.bfloat16, device="cuda"), EPS)
    within(rw, rstdw, rel * rstdw, "rstd")
    within(Yw, yw, (P.BF16 + 3 * rel) * yw.abs(), "Y")


@pytest.mark.parametrize("T,D", [(5, 512), (3, 5120), (1500, 2048), (9000, 512)])
def test_rmsnorm_in_place(T, D):
    X, e = P.random_bf16((T, D), 1.0, 8), P.random_bf16((T, D), 2.0, 9)
    w = P.random_bf16((D,), 1.0, 10)
    Y, H, _ = ops.rmsnorm(X, w, EPS, res=e)
    X2, e2 = X.clone(), e.clone()
    Y2, H2, _ = ops.rmsnorm(X2, w, EPS, res=e2, H=e2, Y=X2)
    assert Y2 is X2 and H2 is e2 and torch.equal(Y2, Y) and torch.equal(H2, H)


# ------------------------------------------------------------------ gradients of the norm
@pytest.mark.parametrize("T,D", NORM_SHAPES + [(2500, 256), (1500, 2048), (1024, 264), (1025, 264), (1024, 5128), (1026, 12288), (1500, 12296), (1100, 18432), (1030, 16384), (1030, 18440),
                                                 (777, 1000), (64, 1032), (300, 20000)])
@pytest.mark.parametrize("dres", [False, True])
def test_rmsnorm_bwd(T, D, dres):
    H, dY = P.random_bf16((T, D), 2.0, 11), P.random_bf16((T, D), 1e-2, 12)
    w = (1 + P.random_bf16((D,), 0.2, 13).float()).to(torch.bfloat16)
    e = P.random_bf16((T, D), 1e-2, 14) if dres else None
    rstd = (H.double().square().mean(1) + EPS).rsqrt().float()
    dH, dw = ops.rmsnorm_bwd(dY, H, w, rstd, dres=e)
    dh, dwr, mag, dwmag = P.norm_bwd(dY, H, w, rstd, e)
    rel = (depth(D) + 10) * P.F32  # the mean's sum, and the ten operations around it
    within(dH, dh, P.BF16 * (dh.abs() + rel * mag) + rel * mag, "dH")
    # dw: a thread's rows in turn, up to eight warps, the parts in eight chains, eight sums, and two products (in one
    # launch: a thread's rows, three shuffles, up to 32 warps, two products)
    chain = -(-T // 64) + 8 + 592 // 8 + 8 + 2
    within(dw, dwr, chain * P.F32 * dwmag, "dw")
    dH2, dw2 = ops.rmsnorm_bwd(dY, H, w, rstd, dres=e)
    assert torch.equal(dH, dH2) and torch.equal(dw, dw2)
    if dres:
        e2 = e.clone()
        dH3, _ = ops.rmsnorm_bwd(dY, H, w, rstd, dres=e2, dH=e2)
        assert torch.equal(dH, dH3)


def test_rmsnorm_bwd_matches_differences_of_the_forward():
    """The call's gradient against differences of the call's own forward, along random directions.  The forward rounds
    Y to bf16, so its difference quotient over a step a is off by up to 2 2^-8 sum |c y| / (2 a) in the worst case."""
    T, D = 4, 256
    H, w = P.random_bf16((T, D), 1.0, 15), (1 + P.random_bf16((D,), 0.2, 16).float()).to(torch.bfloat16)
    c = P.random_bf16((T, D), 1.0, 17)
    Y, _, rstd = ops.rmsnorm(H, w, EPS, with_rstd=True)
    dH, dw = ops.rmsnorm_bwd(c, H, w, rstd)
    a = 0.25
    v = torch.sign(P.random_bf16((T, D), 1.0, 18).float())
    up, down = (H.float() + a * v).to(torch.bfloat16), (H.float() - a * v).to(torch.bfloat16)
    step = up.double() - down.double()
    loss = lambda x: (ops.rmsnorm(x, w, EPS)[0].double() * c.double()).sum()  # noqa: E731
    _, yu, _, _, _ = P.norm(up, w, EPS)
    _, yd, _, _, _ = P.norm(down, w, EPS)
    exact = ((yu - yd) * c.double()).sum()
    noise = P.BF16 * ((yu.abs() + yd.abs()) * c.double().abs()).sum()
    assert abs(loss(up) - loss(down) - exact) <= 1.01 * noise
    # the derivative along the step, against the exact difference: what is left is the curvature, third order in a
    lin = (dH.double() * step).sum()
    third = abs(exact - (P.norm_bwd(c, H, w, rstd)[0] * step).sum())
    assert abs(lin - exact) <= third + P.BF16 * (dH.double() * step).abs().sum() * 1.01


# ------------------------------------------------------------------ product
def product_case(T, K, M, r, seed=0):
    Xq, Wq = P.random_int8(T, K, seed + 1), P.random_int8(M, K // 2, seed + 2)
    g = torch.Generator().manual_seed(seed + 3)
    xs = (torch.rand(T, generator=g) * 0.02 + 0.001).cuda()
    ws = (torch.rand(M, generator=g) * 0.0002 + 0.00001).cuda()
    meta = P.random_codes(M, K, seed + 4)
    XL = P.random_bf16((T, r), 1.0, seed + 5) if r else None
    R = P.random_bf16((r, M), 0.1, seed + 6) if r else None
    return Xq, xs, Wq, ws, meta, XL, R


PRODUCT = [
    # a few tokens: CUDA cores
    (1, 64, 64, 8), (1, 64, 128, 0), (2, 128, 64, 8), (3, 1024, 192, 24), (4, 1088, 448, 96), (1, 9216, 512, 96), (4, 2112, 9536, 16),
    (2, 36864, 128, 0), (4, 65536, 128, 8), (1, 131072, 64, 8), (1, 1024, 20032, 256),
    # 64 channels: half a tile of them
    (5, 192, 64, 8), (37, 4096, 64, 200), (1000, 64, 64, 0), (300, 17024, 64, 256), (16, 256, 64, 16), (3000, 1024, 64, 8), (6, 131072, 64, 24),
    # tensor cores: token tiles of 16, 32, 64, 128, ragged ends in tokens, channels and the sum
    (5, 64, 128, 8), (16, 256, 128, 0), (13, 4096, 192, 96), (17, 512, 320, 16), (32, 1024, 256, 256), (33, 384, 512, 40), (64, 2048, 640, 64),
    (65, 128, 192, 8), (128, 512, 128, 0), (200, 640, 1088, 24), (129, 9216, 256, 96), (1000, 768, 832, 64),
    # codes that TMA cannot load (K an odd multiple of 64)
    (9, 192, 128, 8), (40, 832, 320, 72), (300, 4160, 192, 0), (8, 12352, 256, 16), (5, 64, 256, 8), (20, 320, 3200, 200),
    (100, 5824, 1088, 40), (2500, 64, 640, 8), (3300, 832, 1984, 200), (4000, 1472, 2752, 64), (2222, 5824, 960, 0),
    # long sums on few tiles: split over clusters of up to eight CTAs
    (16, 36864, 256, 96), (8, 131072, 128, 8), (48, 16384, 384, 8), (100, 8192, 128, 64), (12, 2048, 128, 0),
    # many tiles
    (24, 512, 40000, 8), (700, 1024, 5120, 96), (2100, 1536, 2048, 16), (4096, 512, 512, 8),
    # 512 x 224 pair tiles: ragged in channels (clamped blocks), tokens and the sum; every count of adapter k-tiles
    (5000, 128, 128, 0), (4100, 256, 192, 8), (2300, 640, 1088, 256), (1792, 1024, 2560, 96), (3001, 1408, 832, 136), (2048, 2048, 4096, 0),
    (9000, 384, 704, 64), (8000, 2048, 4096, 0), (4501, 4096, 5120, 96), (6000, 832, 5184, 0), (8100, 1984, 4160, 0), (350, 9216, 5184, 256), (256, 4160, 5120, 0),
    # every width at every split
    (500, 1024, 320, 64), (300, 2048, 192, 64), (151, 4096, 192, 64), (501, 1024, 640, 64), (500, 2048, 320, 64), (299, 4096, 192, 64),
    (1000, 1536, 640, 64), (503, 2048, 640, 64), (500, 4096, 320, 64),
    (250, 3328, 320, 64), (499, 3328, 320, 64), (250, 16384, 192, 64), (1000, 2048, 640, 64), (1000, 5120, 320, 64), (500, 16384, 192, 64),
    (1000, 3328, 640, 64), (11, 3392, 192, 40), (13, 5120, 5120, 64),
]


def test_the_cases_cover_every_form():
    forms = {ops.q8_plan(M, T, K, r) for T, K, M, r in PRODUCT}
    assert {f[:2] for f in forms} >= {(0, 1), (0, 2), (0, 4), (128, 16), (128, 32), (128, 64), (128, 128), (256, 256), (512, 224)}
    assert {f[1:] for f in forms if f[0] == 128} == {(bn, s) for bn in (16, 32, 64, 128) for s in (1, 2, 3, 4, 8)}
    odd = {ops.q8_plan(M, T, K, r)[0] for T, K, M, r in PRODUCT if K % 128}
    assert odd == {0, 128, 256, 512}
    assert {ops.q8_plan(M, T, K, r)[0] for T, K, M, r in PRODUCT if M == 64} == {0, 128}


@pytest.mark.parametrize("T,K,M,r", PRODUCT)
def test_fwd_q8(T, K, M, r):
    case = product_case(T, K, M, r)
    Y = ops.fwd_q8(*case, M, Y=guarded_empty((T, M), torch.bfloat16))
    ops.status_sync()
    want, tol = P.product(*case)
    within(Y, want, tol, "Y")
    check_guards()
    Y2 = ops.fwd_q8(*case, M)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("T", [1, 4, 16, 100, 600])
def test_fwd_q8_extreme_values(T):
    """All -128 and all 127, every code equal: the largest sums, exact in 32 bits."""
    K, M = 36864, 256
    Xq, Wq = torch.full((T, K), -128, dtype=torch.int8, device="cuda"), torch.full((M, K // 2), -128, dtype=torch.int8, device="cuda")
    Wq[1::2] = 127
    xs, ws = torch.ones(T, device="cuda"), torch.ones(M, device="cuda")
    for code in P.CODES:
        word = code * 0x1111
        meta = torch.full((M, K // 16), word - 0x10000 if word >= 0x8000 else word, dtype=torch.int16, device="cuda")
        Y = ops.fwd_q8(Xq, xs, Wq, ws, meta, None, None, M)
        want = torch.full((T, M), 128.0 * 128 * K / 2, device="cuda", dtype=torch.float64)
        want[:, 1::2] = -128.0 * 127 * K / 2
        assert torch.equal(Y, want.to(torch.bfloat16))


@pytest.mark.parametrize("T", [1, 16, 300, 1500])
def test_fwd_q8_scales_of_zero_and_nan(T):
    K, M, r = 512, 320, 16
    Xq, xs, Wq, ws, meta, XL, R = product_case(T, K, M, r)
    xs[T // 2] = float("nan")
    ws[7] = float("nan")
    ws[9] = 0
    ws[M - 1] = float("inf")
    Xq[0] = 0
    if T > 1:
        xs[0] = 0
    Y = ops.fwd_q8(Xq, xs, Wq, ws, meta, XL, R, M)
    want, tol = P.product(Xq, xs, Wq, ws, meta, XL, R)
    bad = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(Y), torch.isnan(want))
    assert torch.equal(torch.where(bad, 0.0, Y.double()).isinf(), torch.zeros_like(bad))
    within(torch.where(bad, 0.0, Y.double()), torch.where(bad, 0.0, want), torch.where(bad, 0.0, tol), "Y")


def test_adapter_alone_where_the_tokens_are_zero():
    T, K, M, r = 40, 256, 256, 64
    Xq, xs, Wq, ws, meta, XL, R = product_case(T, K, M, r)
    Xq.zero_()
    xs.zero_()
    Y = ops.fwd_q8(Xq, xs, Wq, ws, meta, XL, R, M)
    want, tol = P.product(Xq, xs, Wq, ws, meta, XL, R)
    within(Y, want, tol, "Y")


# ------------------------------------------------------------------ as they are used together
def chain(X, res, wn, W, L, R, out):
    """The layer as an int8 user runs it: prune and quantise once, then norm, down-projection, product."""
    vals, meta = ops.prune24(W)
    vq, ws = ops.quant_rows(vals)
    Q, s, Y, H, _ = ops.rmsnorm_q8(X, wn, EPS, res=res, with_y=True)
    XL = ops.adapter_fwd(Y, L)
    return (vals, meta, vq, ws, Q, s, Y, H, XL), ops.fwd_q8(Q, s, vq, ws, meta, XL, R, out)


@pytest.mark.parametrize("T,inn,out,r", [(1, 768, 512, 16), (16, 1024, 1024, 64), (300, 512, 640, 16), (1200, 1024, 1536, 96)])
def test_layer_in_int8(T, inn, out, r):
    X, e = P.random_bf16((T, inn), 1.0, 21), P.random_bf16((T, inn), 2.0, 22)
    wn = (1 + P.random_bf16((inn,), 0.2, 23).float()).to(torch.bfloat16)
    W, L, R = P.random_bf16((out, inn), 0.02, 24), P.random_bf16((inn, r), 0.02, 25), P.random_bf16((r, out), 0.02, 26)
    (vals, meta, vq, ws, Q, s, Yn, H, XL), Y = chain(X, e, wn, W, L, R, out)
    ops.status_sync()
    h, y, _, q, _ = P.norm(X, wn, EPS, e)
    assert torch.equal(H, h) and torch.equal(Q, q)
    qw, _ = P.quantise(vals.double())
    assert torch.equal(vq, qw)
    want, tol = P.product(Q, s, vq, ws, meta, XL, R)
    within(Y, want, tol, "Y")
    # and against the bf16 layer: quantising moves a value by at most half a step, s / 2 for a token, ws / 2 for a weight
    Wd, nd = P.dense(vals, meta, inn), Yn.double()
    half_x, half_w = s.double()[:, None] / 2, ws.double() / 2
    kept = (P.dense(torch.ones_like(vals), meta, inn)).t()
    bound = (half_x + P.BF16 * nd.abs()) @ Wd.t().abs() + ((nd.abs() + half_x) @ kept) * half_w
    exact = nd @ Wd.t() + XL.double() @ R.double()
    assert ((Y.double() - exact).abs() <= 1.01 * bound + tol + 1e-6).all()


@pytest.mark.parametrize("T", [1, 16, 300, 1200])
def test_captured_and_replayed(T):
    """The whole chain in a CUDA graph, replayed on new tokens, beside eager calls; two graphs share nothing."""
    inn, out, r = 1024, 1536, 64
    wn = (1 + P.random_bf16((inn,), 0.2, 23).float()).to(torch.bfloat16)
    W, L, R = P.random_bf16((out, inn), 0.02, 24), P.random_bf16((inn, r), 0.02, 25), P.random_bf16((r, out), 0.02, 26)
    vals, meta = ops.prune24(W)
    vq, ws = ops.quant_rows(vals)
    X, e = P.random_bf16((T, inn), 1.0, 21), P.random_bf16((T, inn), 2.0, 22)
    XL = P.random_bf16((T, r), 1.0, 27)
    dY = P.random_bf16((T, inn), 1e-2, 28)

    def step(X, e):
        Q, s, Y, H, rstd = ops.rmsnorm_q8(X, wn, EPS, res=e, with_y=True, with_rstd=True)
        dH, dw = ops.rmsnorm_bwd(dY, H, wn, rstd, dres=e)
        return ops.fwd_q8(Q, s, vq, ws, meta, XL, R, out), dH, dw
    step(X, e)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        Xg, eg = torch.zeros_like(X), torch.zeros_like(e)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step(Xg, eg)
        graphs.append((g, Xg, eg, got))
    for k, (g, Xg, eg, got) in enumerate(graphs):
        Xg.copy_(X * (k + 1))
        eg.copy_(e)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for (g, *_), st in zip(graphs, streams):
        with torch.cuda.stream(st):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for k, (g, Xg, eg, got) in enumerate(graphs):
        for a, b in zip(got, step(Xg, eg)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,M", [(2, 2048, 1024), (16, 8192, 512), (300, 1024, 1024), (1500, 1024, 2048)])
def test_calls_on_several_streams_overlap_safely(T, K, M):
    cases = [product_case(T, K, M, 16, seed=100 * i) for i in range(4)]
    want = [ops.fwd_q8(*c, M) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(ops.fwd_q8(*c, M))
    torch.cuda.synchronize()
    ops.status_sync()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4])


def test_offsets_past_32_bits():
    """More than 2^31 values in every operand: the last rows are the right ones (the first ones' neighbours would be
    overwritten by an offset that wrapped)."""
    rows, K = 262200, 8208
    tail = 3
    A = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    A[-tail:] = P.random_bf16((tail, K), 1.0, 41)
    Q, scale = ops.quant_rows(A)
    q, top = P.quantise(A[-tail:].double())
    assert torch.equal(Q[-tail:], q) and not Q[:5].any() and not scale[:-tail].any()
    w = (1 + P.random_bf16((K,), 0.2, 42).float()).to(torch.bfloat16)
    Q, _, Y, H, rstd = ops.rmsnorm_q8(A, w, EPS, res=A, with_y=True, with_rstd=True)
    h, y, _, q, _ = P.norm(A[-tail:], w, EPS, A[-tail:])
    assert torch.equal(H[-tail:], h) and torch.equal(Q[-tail:], q) and not Y[:5].any()
    within(Y[-tail:], y, P.BF16 * 1.01 * y.abs(), "Y")
    del Q, Y
    dH, dw = ops.rmsnorm_bwd(A, H, w, rstd)
    dh, dwr, mag, dwmag = P.norm_bwd(A[-tail:], h, w, rstd[-tail:])
    within(dH[-tail:], dh, P.BF16 * dh.abs() + 2.0 ** -17 * mag, "dH")
    within(dw, dwr, 8 * P.F32 * dwmag, "dw")  # every other row adds zeros
    del A, H, dH
    for T, K, M in ((1 << 15, 128, 65600), (1 << 15, 64, 65600)):  # Y has 2^31 values and some
        Xq, xs, Wq, ws, meta, XL, R = product_case(8, K, M, 8)
        X = torch.zeros(T, K, dtype=torch.int8, device="cuda")
        X[-8:] = Xq
        s = torch.zeros(T, device="cuda")
        s[-8:] = xs
        L = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
        L[-8:] = XL
        Y = ops.fwd_q8(X, s, Wq, ws, meta, L, R, M)
        want, tol = P.product(Xq, xs, Wq, ws, meta, XL, R)
        within(Y[-8:], want, tol, "Y")
        assert not Y[:40].any()


def test_captured_before_any_call():
    """A process whose first calls are captured: set-up that a warm-up would have done works during capture."""
    import subprocess
    import sys
    code = """
import sys, torch
sys.path.insert(0, 'tests')
import q8_plain as P
from structured_sparse_pretraining_b200 import ops
T, K, M, r = 1500, 1280, 640, 16
X, w = P.random_bf16((T, K), 1.0, 1), P.random_bf16((K,), 1.0, 2)
A = P.random_bf16((M, K // 2), 0.02, 3)
meta, XL, R = P.random_codes(M, K, 4), P.random_bf16((T, r), 1.0, 5), P.random_bf16((r, M), 0.1, 6)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    vq, ws = ops.quant_rows(A)
    Q, s, Y, _, rstd = ops.rmsnorm_q8(X, w, 1e-5, with_y=True, with_rstd=True)
    dH, dw = ops.rmsnorm_bwd(Y, X, w, rstd)
    out = [ops.fwd_q8(Q[:t], s[:t], vq, ws, meta, XL[:t], R, M) for t in (1, 16, 200, T)]
g.replay()
torch.cuda.synchronize()
for t, y in zip((1, 16, 200, T), out):
    want, tol = P.product(Q[:t], s[:t], vq, ws, meta, XL[:t], R)
    assert ((y.double() - want).abs() <= tol).all(), t
ops.status_sync()
print('captured first')
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "captured first" in res.stdout, res.stdout[-2000:] + res.stderr[-2000:]


def test_refusals_on_the_gpu():
    X, w = P.random_bf16((4, 64), 1.0, 1), P.random_bf16((64,), 1.0, 2)
    with pytest.raises(ValueError, match="contiguous"):
        ops.rmsnorm(P.random_bf16((64, 4), 1.0, 1).t(), w, EPS)
    with pytest.raises(ValueError, match="shape"):
        ops.rmsnorm(X, w[:56].contiguous(), EPS)
    with pytest.raises(ValueError, match="two dimensions"):
        ops.rmsnorm(X.view(2, 2, 64), w, EPS)
    with pytest.raises(ValueError, match="bfloat16"):
        ops.quant_rows(X.float())
    with pytest.raises(ValueError, match="H without res"):
        ops.rmsnorm(X, w, EPS, H=torch.empty_like(X))
    with pytest.raises(Exception, match="SLOPE_ERR_ARG"):
        ops.rmsnorm(X, w, 0.0)
    with pytest.raises(Exception, match="SLOPE_ERR_SHAPE"):
        ops.quant_rows(P.random_bf16((4, 12), 1.0, 1))
    with pytest.raises(Exception, match="SLOPE_ERR_ARG"):
        ops.rmsnorm(X[:0], w, EPS)
    Xq, xs, Wq, ws, meta, XL, R = product_case(4, 128, 64, 8)
    with pytest.raises(ValueError, match="XL without R"):
        ops.fwd_q8(Xq, xs, Wq, ws, meta, XL, None, 64)
    with pytest.raises(ValueError, match="vals_q"):
        ops.fwd_q8(Xq, xs, Wq[:, :32].contiguous(), ws, meta, XL, R, 64)
    with pytest.raises(ValueError, match="int8"):
        ops.fwd_q8(Xq.float(), xs, Wq, ws, meta, XL, R, 64)


@pytest.mark.parametrize("T,D", [(9, 264), (5, 5120), (1201, 1544), (8001, 520)])
def test_no_writes_outside_outputs(T, D):
    X, e, w = P.random_bf16((T, D), 1.0, 1), P.random_bf16((T, D), 1.0, 2), P.random_bf16((D,), 1.0, 3)
    G = lambda shape, t: guarded_empty(shape, t)  # noqa: E731
    _CANARY.setdefault(torch.int8, 0x25)
    H, Y, s, rs = G((T, D), torch.bfloat16), G((T, D), torch.bfloat16), G((T,), torch.float32), G((T,), torch.float32)
    Q = guarded_empty((T, D), torch.uint8).view(torch.int8)
    ops.rmsnorm_q8(X, w, EPS, res=e, H=H, Y=Y, Q=Q, qscale=s, rstd=rs)
    ops.rmsnorm_bwd(X, H, w, rs, dres=e, dH=G((T, D), torch.bfloat16), dw=G((D,), torch.float32))
    ops.quant_rows(X, Q=guarded_empty((T, D), torch.uint8).view(torch.int8), scale=G((T,), torch.float32))
    ops.status_sync()
    check_guards()
