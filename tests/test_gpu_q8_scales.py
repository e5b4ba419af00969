"""fwd_q8 with scales whose product leaves binary32's range, in every form of the launch."""
import pytest
import torch

import q8_plain as P
from structured_sparse_pretraining_b200 import ops

pytestmark = pytest.mark.gpu
# CUDA cores, 128-row tiles alone and in clusters, 256-row and 512-row tiles
SHAPES = [(1, 512, 320, 0), (3, 1024, 192, 8), (16, 256, 128, 16), (16, 36864, 256, 96), (100, 832, 320, 24),
          (300, 4160, 9216, 0), (512, 4096, 5120, 64), (3300, 832, 1984, 200), (5000, 128, 128, 0), (2048, 2048, 4096, 8)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    ops.device_check()
    yield
    ops.status_sync()


def operands(T, K, M, r):
    Xq, Wq, meta = P.random_int8(T, K, 1), P.random_int8(M, K // 2, 2), P.random_codes(M, K, 3)
    return Xq, Wq, meta, P.random_bf16((T, r), 1.0, 4) if r else None, P.random_bf16((r, M), 0.1, 5) if r else None


def test_the_shapes_cover_every_form():
    assert {ops.q8_plan(M, T, K, r)[0] for T, K, M, r in SHAPES} == {0, 128, 256, 512}


@pytest.mark.parametrize("T,K,M,r", SHAPES)
def test_zero_sums_under_large_scales(T, K, M, r):
    """A sum of zero stays zero, whatever finite scales say."""
    Xq, Wq, meta, XL, R = operands(T, K, M, r)
    Xq.zero_()
    xs, ws = torch.full((T,), 2.0 ** 90, device="cuda"), torch.full((M,), 2.0 ** 60, device="cuda")
    Y = ops.fwd_q8(Xq, xs, Wq, ws, meta, XL, R, M)
    want, tol = P.product(Xq, xs, Wq, ws, meta, XL, R)
    assert ((Y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("T,K,M,r", SHAPES)
def test_scales_whose_product_is_subnormal(T, K, M, r):
    Xq, Wq, meta, _, _ = operands(T, K, M, 0)
    xs, ws = 1.37 * torch.full((T,), 2.0 ** -83, device="cuda"), 1.71 * torch.full((M,), 2.0 ** -64, device="cuda")
    Y = ops.fwd_q8(Xq, xs, Wq, ws, meta, None, None, M)
    want, tol = P.product(Xq, xs, Wq, ws, meta)
    # the last places of subnormals, bf16's 2^-133 and binary32's 2^-149
    assert ((Y.double() - want).abs() <= tol + 2.0 ** -134 + 2.0 ** -149).all()


@pytest.mark.parametrize("T,K,M,r", [(1, 512, 320, 256), (16, 256, 128, 256), (100, 832, 320, 256), (512, 4096, 5120, 256), (300, 4160, 9216, 128),
                                     (3300, 832, 1984, 256), (2048, 2048, 4096, 256)])
def test_adapter_that_cancels_the_sum(T, K, M, r):
    """XL . R close to minus the int8 term, its parts spread over the whole rank: what is left shows every rounding.
    The sum's part takes four roundings, and in the forms of 256 and 512 rows two units more for each 16 of the rank."""
    Xq, Wq, meta, _, _ = operands(T, K, M, 0)
    Xq = Xq[:r].repeat(-(-T // r), 1)[:T].contiguous()  # token t repeats token t % r
    xs = torch.full((T,), 1.37 / 64, device="cuda")
    ws = torch.rand(M, generator=torch.Generator().manual_seed(7)).cuda() * 0.01 + 0.001
    main, _ = P.product(Xq, xs, Wq, ws, meta)
    H = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while H.shape[0] < r:  # Hadamard: rows of +-1, H H^T = r
        H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)], 0)
    base = torch.zeros(r, M, dtype=torch.float64, device="cuda")
    base[:min(T, r)] = main[:r]
    R = (-(H.t() @ base) / r).to(torch.bfloat16)
    XL = H.to(torch.bfloat16).repeat(-(-T // r), 1)[:T].contiguous()
    Y = ops.fwd_q8(Xq, xs, Wq, ws, meta, XL, R, M)
    mags = XL.double().abs() @ R.double().abs()
    want = main + XL.double() @ R.double()
    assert want.abs().mean() < 0.02 * main.abs().mean(), "the terms cancel"
    joined = ops.q8_plan(M, T, K, r)[0] <= 128
    slack = (4 if joined else 4 + 2 * -(-r // 16)) * P.F32 * main.abs() + 2 * (r + 2) * P.F32 * mags
    assert ((Y.double() - want).abs() <= P.BF16 * want.abs() + (1 + P.BF16) * slack).all()
