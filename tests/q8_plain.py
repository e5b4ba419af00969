"""Plain 64-bit forms of the int8 path's operators, for its tests.

Rounding units used by the tolerances: a bf16 result is off by at most 2^-8 of
its value, a binary32 operation by 2^-24 of its result.  A sum of n binary32
terms added in any order is off by at most (n - 1) 2^-24 times the sum of
their magnitudes; the sums here are trees, so `depth` below counts the
additions on the longest path from a term to the result.
"""
import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24
CODES = (0x4, 0x8, 0xC, 0x9, 0xD, 0xE)


def quantise(p):
    """round(127 p / max |p|) per row, ties to even, and max |p|; p in 64 bits.  A row with a value that is not finite gives 0."""
    top = p.abs().amax(1, keepdim=True)
    ok = torch.isfinite(p).all(1, keepdim=True) & (top > 0)
    q = torch.where(ok, torch.round(127.0 * torch.where(ok, p, 0.0) / torch.where(ok, top, 1.0)), 0.0)
    return q.to(torch.int8), torch.where(torch.isfinite(p).all(1), top[:, 0], float("nan"))


def norm(X, w, eps, res=None):
    """(h bf16, y, rstd, Q, qscale): the norm of rows, 64 bits but for h."""
    h = X if res is None else (X.float() + res.float()).to(torch.bfloat16)
    hd, wd = h.double(), w.double()
    rstd = (hd.square().mean(1) + eps).rsqrt()
    Q, top = quantise(hd * wd)
    return h, hd * rstd[:, None] * wd, rstd, Q, rstd * top / 127


def norm_bwd(dY, h, w, rstd, dres=None):
    """(dh, dw) and the magnitudes the roundings of each act on."""
    dY, h, w, rstd = dY.double(), h.double(), w.double(), rstd.double()[:, None]
    n, g = h * rstd, dY * w
    mean, amean = (g * n).mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
    dh = rstd * (g - n * mean)
    mag = rstd * (g.abs() + n.abs() * amean)
    if dres is not None:
        dh, mag = dh + dres.double(), mag + dres.double().abs()
    return dh, (dY * n).sum(0), mag, (dY * n).abs().sum(0)


def dense(vals, meta, K):
    """The dense [rows, K] 64-bit matrix of a 2:4-compressed one."""
    rows = vals.shape[0]
    out = torch.zeros(rows, K // 4, 4, dtype=torch.float64, device=vals.device)
    word = meta.to(torch.int64) & 0xFFFF
    for j in range(8):
        place = ((word >> (2 * j)) & 3)
        g = torch.arange(K // 16, device=vals.device) * 4 + j // 2
        out[torch.arange(rows, device=vals.device)[:, None], g[None, :], place] = vals.view(rows, K // 16, 8)[:, :, j].double()
    return out.view(rows, K)


def product(Xq, xscale, vals_q, wscale, meta, XL=None, R=None):
    """(Y, its tolerance) in 64 bits: int8 sums are exact; the sum, the two scales' product and the join round in
    binary32, the adapter's r products and additions too (tensor cores may truncate: two units), Y once to bf16."""
    main = (Xq.double() @ dense(vals_q, meta, Xq.shape[1]).t()) * xscale.double()[:, None] * wscale.double()
    Y, slack = main, 4 * F32 * main.abs()
    if R is not None:
        Y = main + XL.double() @ R.double()
        slack = slack + 2 * (R.shape[0] + 2) * F32 * (XL.double().abs() @ R.double().abs())
    return Y, BF16 * (Y.abs() + slack) + slack


def random_codes(rows, K, seed, device="cuda"):
    """Random legal code words [rows, K/16] int16."""
    g = torch.Generator().manual_seed(seed)
    c = torch.tensor(CODES, dtype=torch.int32)[torch.randint(0, 6, (rows, K // 16, 4), generator=g)]
    word = c[..., 0] | c[..., 1] << 4 | c[..., 2] << 8 | c[..., 3] << 12
    return torch.where(word >= 0x8000, word - 0x10000, word).to(torch.int16).to(device)


def random_int8(rows, K, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-127, 128, (rows, K), generator=g, dtype=torch.int32).to(torch.int8).to(device)


def random_bf16(shape, std, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(device)
