"""The norm's rows at the ends of binary32's range, against the plain 64-bit form."""
import pytest
import torch

import q8_plain as P
from structured_sparse_pretraining_b200 import ops

pytestmark = pytest.mark.gpu
# rows of a warp, of a CTA, and in the ring of rows
SHAPES = [(5, 256), (5, 1000), (6, 5120), (3, 32768), (1300, 8192)]
F32 = P.F32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    ops.device_check()
    yield
    ops.status_sync()


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol) & ~(got == want)
    assert not bad.any(), f"{what}: {int(bad.sum())} values, first at {bad.nonzero()[0].tolist()}"


def rel(D):
    """rstd's relative error: a sum of up to 74 additions in a row, halved by the root, and six operations."""
    return (74 / 2 + 6) * F32


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("scale,eps", [(2.0 ** 63.5, 1e38), (2.0 ** 63.5, 3.0e38), (2.0 ** 40, 3.4e38), (2.0 ** -72, 2.0 ** -140),
                                       (2.0 ** -100, 2.0 ** -149), (2.0 ** -63, 2.0 ** -126), (2.0 ** -60, 2.0 ** -121)])
def test_eps_beside_sums_outside_the_normal_range(T, D, scale, eps):
    """eps counts where the squares' sum overflows, and where eps itself is subnormal."""
    X = (P.random_bf16((T, D), 1.0, 1).float() * scale).to(torch.bfloat16)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    eps = float(torch.tensor(eps, dtype=torch.float32))
    Y, _, rstd = ops.rmsnorm(X, w, eps, with_rstd=True)
    _, y, want, _, _ = P.norm(X, w, eps)
    close(rstd, want, rel(D) * want, "rstd")
    close(Y, y, (P.BF16 + 3 * rel(D)) * y.abs() + 2.0 ** -134, "Y")


def check_row(X, w, eps, res=None, Y=None):
    h, y, rstd, q, qs = P.norm(X.clone(), w, eps, None if res is None else res.clone())
    D = X.shape[1]
    Q, s, Y, H, rs = ops.rmsnorm_q8(X, w, eps, res=res, with_y=True, with_rstd=True, Y=Y)
    assert torch.equal(Q, q)
    close(rs, rstd, rel(D) * rstd, "rstd")
    close(s, qs, (rel(D) + 3 * F32) * qs + 2.0 ** -150, "qscale")  # half of a subnormal's last place
    # rounded once to binary32 and once to bf16, whose last places end at 2^-149 and 2^-133
    close(Y, y, (P.BF16 * 1.01 + 2 * rel(D)) * y.abs() + 2.0 ** -134 + 2.0 ** -136, "Y")
    if res is not None:
        assert torch.equal(H, h)
    return Q, s, Y


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("hs,ws,eps", [(-72, -76, 1e-5), (-72, -76, 1e-30), (-100, -50, 1e-38), (-126, -126, 1e-5), (-133, -133, 2.0 ** -149),
                                       (-60, -55, 2.0 ** -120), (-3, -130, 1e-6), (60, -133, 1e-5)])
def test_products_below_the_normal_range(T, D, res, hs, ws, eps):
    """Rows whose products h w have bits below binary32's last place: codes are those of the exact products."""
    eps = float(torch.tensor(eps, dtype=torch.float32))
    X = (P.random_bf16((T, D), 1.0, 1).double() * 2.0 ** hs).to(torch.bfloat16)
    e = (P.random_bf16((T, D), 1.0, 2).double() * 2.0 ** hs).to(torch.bfloat16) if res else None
    w = ((1 + 0.2 * P.random_bf16((D,), 1.0, 3).double()) * 2.0 ** ws).to(torch.bfloat16)
    X[1] = 0
    if res:
        e[1] = 0
    X[2] = (X[2].double() * 2.0 ** min(40, 100 - hs)).to(torch.bfloat16)  # an ordinary row beside them
    Q, s, _ = check_row(X, w, eps, e)
    assert Q[0].any() and not Q[1].any() and s[1] == 0
    if T < 10:  # in place
        check_row(X, w, eps, e, Y=X)


def test_products_below_the_normal_range_by_hand():
    h = torch.tensor([[1.0, 0.498046875, 0.25, 0.330078125, 0, 0, 0, 0]], device="cuda") * 2.0 ** -72
    Q, _, _, _, _ = ops.rmsnorm_q8(h.to(torch.bfloat16), torch.full((8,), 2.0 ** -76, device="cuda").to(torch.bfloat16), 1e-5)
    assert Q.tolist() == [[127, 63, 32, 42, 0, 0, 0, 0]]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_small_weights_beside_ordinary_ones(T, D, res):
    """A row in range as a whole, some of whose products are not, with an rstd that brings them back into bf16's range."""
    X = (P.random_bf16((T, D), 1.0, 4).double() * 2.0 ** -40).to(torch.bfloat16)
    e = (P.random_bf16((T, D), 1.0, 5).double() * 2.0 ** -40).to(torch.bfloat16) if res else None
    w = P.random_bf16((D,), 1.0, 6).double()
    w[::3] *= 2.0 ** -100
    check_row(X, w.to(torch.bfloat16), 2.0 ** -100, e)


def test_in_place_where_rows_are_read_again():
    for T, D in SHAPES:
        X = (P.random_bf16((T, D), 1.0, 7).double() * 2.0 ** -70).to(torch.bfloat16)
        e = (P.random_bf16((T, D), 1.0, 8).double() * 2.0 ** -70).to(torch.bfloat16)
        w = (P.random_bf16((D,), 1.0, 9).double() * 2.0 ** -70).to(torch.bfloat16)
        want = ops.rmsnorm_q8(X, w, 1e-30, res=e, with_y=True)
        for h_in, y_in in (("X", "e"), ("e", "X")):
            t = dict(X=X.clone(), e=e.clone())
            got = ops.rmsnorm_q8(t["X"], w, 1e-30, res=t["e"], H=t[h_in], Y=t[y_in])
            for a, b in zip(got[:4], want[:4]):
                assert torch.equal(a, b), (T, D, h_in)
        want = ops.rmsnorm_q8(X, w, 1e-30, with_y=True)
        got = ops.rmsnorm_q8(X, w, 1e-30, Y=X)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_products_above_the_range(T, D, res):
    """h w overflows binary32, h rstd w does not: Y is that; in int8 the row has no scale."""
    X = (P.random_bf16((T, D), 1.0, 1).double() * 2.0 ** 100).to(torch.bfloat16)
    e = (P.random_bf16((T, D), 1.0, 2).double() * 2.0 ** 100).to(torch.bfloat16) if res else None
    w = (P.random_bf16((D,), 1.0, 3).double() * 2.0 ** 40).to(torch.bfloat16)
    X[1], X[2, 5] = 1.0, float("inf")
    if res:
        e[1] = 0.5
    h, y, rstd, _, _ = P.norm(X, w, 1e-5, e)
    for y_only in (True, False):
        if y_only:
            Y, H, rs = ops.rmsnorm(X, w, 1e-5, res=e, with_rstd=True)
        else:
            Q, s, Y, H, rs = ops.rmsnorm_q8(X, w, 1e-5, res=e, with_y=True, with_rstd=True)
            assert torch.isnan(s[[0, 2]]).all() and not Q[[0, 2]].any() and torch.isfinite(s[1]) and Q[1].any()
        rows = [i for i in range(T) if i != 2]
        close(rs[rows], rstd[rows], rel(D) * rstd[rows], "rstd")
        close(Y[rows], y[rows], (P.BF16 * 1.01 + 2 * rel(D)) * y[rows].abs(), "Y")
        assert torch.isfinite(Y[rows].float()).all()
        assert rs[2] == 0 and torch.isnan(Y[2, 5]) and not Y[2, :5].any()
        if res:
            assert torch.equal(H, h)


@pytest.mark.parametrize("T,D", SHAPES)
def test_scale_of_outputs_above_the_range(T, D):
    """One value carries each row, so rstd h is about sqrt(D); with w near the end of the range h rstd w overflows, its
    127th part, the scale, does not."""
    X = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    X[:, 3] = 2.0
    w = torch.full((D,), 2.0 ** 126, device="cuda").to(torch.bfloat16)
    Q, s, _, _, _ = ops.rmsnorm_q8(X, w, 1e-5)
    _, _, _, q, qs = P.norm(X, w, 1e-5)
    assert torch.equal(Q, q) and torch.isfinite(s).all()
    close(s, qs, (rel(D) + 3 * F32) * qs, "qscale")
