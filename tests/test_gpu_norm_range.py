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
