"""The int8 inference path of the sparse layer and the normalisation before it, as measured cases.

Four operators:

  norm      root-mean-square norm of the tokens entering a linear, with the residual stream's addition, and its
            output in bf16 (for the bf16 products and the adapter), in int8 with one scale per token (for the
            int8 product), or both
  norm_bwd  its gradients: of the tokens (with the gradient that arrives along the residual stream) and of the weight
  quant     int8 quantisation of rows with one scale per row: the kept weights of a 2:4-compressed matrix (a row is
            an output channel) or tokens that no norm produced
  product   the sparse linear in int8: Y = xscale wscale (Xq . Wq^T) + XL . R, with Wq the 2:4-compressed int8
            weights, one scale per token and one per output channel, and the bf16 rank-r adapter

`run` computes them in plain torch operations, or where `own` is set through the package's public calls.
"""
import math

import torch

own = False

EPS = 1e-5
CODES = (0x4, 0x8, 0xC, 0x9, 0xD, 0xE)  # the six legal position codes i0 | i1 << 2, i0 < i1


def listed():
    return [
        # one token of a decode step entering the int8 QKV product of the OPT-66B-shaped layer: latency
        dict(name="norm_decode_1x9216", op="norm", T=1, D=9216, res=True, y=True, q8=True, rstd=False, pad=0),
        # the norm of a training batch of the OPT-13B-shaped layer, statistics kept for its backward pass
        dict(name="norm_train_8192x5120", op="norm", T=8192, D=5120, res=True, y=True, q8=False, rstd=True, pad=0),
        # a ragged padded batch of a small model (768 features), first layer: no residual yet
        dict(name="norm_ragged_1027x768", op="norm", T=1027, D=768, res=False, y=False, q8=True, rstd=False, pad=19),
        # prefill of the OPT-66B-shaped layer: int8 for the product, bf16 for the adapter's down-projection
        dict(name="norm_prefill_8192x9216", op="norm", T=8192, D=9216, res=True, y=True, q8=True, rstd=False, pad=0),
        # the backward pass of the training batch above, the residual stream's gradient added
        dict(name="normbwd_train_8192x5120", op="norm_bwd", T=8192, D=5120, dres=True),
        # an odd width and a ragged token count
        dict(name="normbwd_odd_777x1000", op="norm_bwd", T=777, D=1000, dres=False),
        # the kept weights of the OPT-66B-shaped QKV layer, once after loading a checkpoint
        dict(name="quant_weights_27648x4608", op="quant", rows=27648, K=4608, pad=0),
        # sixteen tokens between the two feed-forward linears
        dict(name="quant_tokens_16x36864", op="quant", rows=16, K=36864, pad=1),
        # one token through the QKV layer: the weights are streamed once
        dict(name="product_decode_1_9216_27648", op="product", T=1, K=9216, N=27648, r=96),
        # a decode batch of sixteen through the second feed-forward layer: a long sum, few output channels
        dict(name="product_batch_16_36864_9216", op="product", T=16, K=36864, N=9216, r=96),
        # a ragged prefill of a BERT-Large-shaped feed-forward layer without an adapter
        dict(name="product_ragged_333_1024_4096", op="product", T=333, K=1024, N=4096, r=0),
        # a full prefill batch through the first feed-forward layer of the OPT-66B-shaped model
        dict(name="product_prefill_8192_9216_36864", op="product", T=8192, K=9216, N=36864, r=96),
    ]


def _logint(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "product", "product"])
    if op in ("norm", "norm_bwd"):
        D = _logint(rng, 64, 16384, 8)
        T = _logint(rng, 1, min(16384, (8192 * 9216) // D))
        if op == "norm_bwd":
            return dict(op=op, T=T, D=D, dres=rng.random() < 0.5)
        y, q8 = rng.choice([(True, True), (True, False), (False, True)])
        return dict(op=op, T=T, D=D, res=rng.random() < 0.6, y=y, q8=q8, rstd=rng.random() < 0.5,
                    pad=rng.randint(0, min(T - 1, 9)))
    if op == "quant":
        K = _logint(rng, 64, 36864, 16)
        rows = _logint(rng, 1, min(36864, (36864 * 9216) // (2 * K)))
        return dict(op=op, rows=rows, K=K, pad=rng.randint(0, min(rows - 1, 9)))
    K = _logint(rng, 64, 36864, 64)
    N = _logint(rng, 64, min(36864, (36864 * 9216) // K // 64 * 64), 64)
    T = _logint(rng, 1, 8192)
    r = rng.choice([0, 8, 16, 24, 64, 96, 128, 200, 256])
    return dict(op=op, T=T, K=K, N=N, r=r)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _int8(g, rows, K, std):
    """Rows of normal values in int8 with their scales, and no zero among the scales."""
    v = torch.randn((rows, K), generator=g, device="cuda")
    top = v.abs().amax(1, keepdim=True)
    return (v * (127.0 / top)).round_().to(torch.int8), (top[:, 0] * (std / 127.0)).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "norm":
        T, D = case["T"], case["D"]
        s = dict(X=_normal(g, (T, D)), res=_normal(g, (T, D), 2.0) if case["res"] else None,
                 w=(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16))
        if case["pad"]:  # padding tokens at the end of the batch
            s["X"][T - case["pad"]:] = 0
            if case["res"]:
                s["res"][T - case["pad"]:] = 0
    elif op == "norm_bwd":
        T, D = case["T"], case["D"]
        H = _normal(g, (T, D), 2.0)
        s = dict(dY=_normal(g, (T, D), 1e-2), H=H, w=(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16),
                 rstd=torch.rsqrt(H.float().square().mean(1) + EPS), dres=_normal(g, (T, D), 1e-2) if case["dres"] else None)
    elif op == "quant":
        s = dict(A=_normal(g, (case["rows"], case["K"]), 0.02))
        if case["pad"]:
            s["A"][case["rows"] - case["pad"]:] = 0
    else:
        T, K, N, r = case["T"], case["K"], case["N"], case["r"]
        Xq, xs = _int8(g, T, K, 1.0)
        Wq, ws = _int8(g, N, K // 2, 0.02)
        pick = torch.randint(0, 6, (N, K // 4), generator=g, device="cuda", dtype=torch.uint8)
        code = torch.tensor(CODES, dtype=torch.int16, device="cuda")[pick.int()].view(N, K // 16, 4)
        meta = code[..., 0] | (code[..., 1] << 4) | (code[..., 2] << 8) | (code[..., 3] << 12)
        s = dict(Xq=Xq, xs=xs, Wq=Wq, ws=ws, meta=meta.contiguous(), XL=_normal(g, (T, r)) if r else None,
                 R=_normal(g, (r, N), 0.1) if r else None)
    s["case"] = dict(case)
    return s


def _run_own(s):
    from structured_sparse_pretraining_b200 import ops

    case = s["case"]
    if case["op"] == "norm":
        if case["q8"]:
            Q, qscale, Y, H, rstd = ops.rmsnorm_q8(s["X"], s["w"], EPS, res=s["res"], with_y=case["y"], with_rstd=case["rstd"])
        else:
            Q, qscale = None, None
            Y, H, rstd = ops.rmsnorm(s["X"], s["w"], EPS, res=s["res"], with_rstd=case["rstd"])
        return {"H": H, "Y": Y, "Q": Q, "qscale": qscale, "rstd": rstd}
    if case["op"] == "norm_bwd":
        dH, dw = ops.rmsnorm_bwd(s["dY"], s["H"], s["w"], s["rstd"], dres=s["dres"])
        return {"dH": dH, "dw": dw}
    if case["op"] == "quant":
        Q, scale = ops.quant_rows(s["A"])
        return {"Q": Q, "scale": scale}
    return {"Y": ops.fwd_q8(s["Xq"], s["xs"], s["Wq"], s["ws"], s["meta"], s["XL"], s["R"], case["N"])}


def _codes(meta):
    """Position codes [N, K/4] of the words [N, K/16]."""
    shift = torch.arange(0, 16, 4, device=meta.device, dtype=torch.int32)
    return ((meta.int().unsqueeze(-1) >> shift) & 15).view(meta.shape[0], -1)


def _quantised(p):
    """Rows of p in int8: round(127 p / max |p|), ties to even, taken in 64 bits (values beside a border); the
    largest magnitudes. A row of zeros gives zeros."""
    top = p.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(127.0 * p.double() / top.double()), 0.0)
    return q.to(torch.int8), top[:, 0]


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "norm":
        H = (s["X"].float() + s["res"].float()).to(torch.bfloat16) if case["res"] else None
        h, w = (H if case["res"] else s["X"]).float(), s["w"].float()
        rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
        Y = (h * rstd[:, None] * w).to(torch.bfloat16) if case["y"] else None
        Q, top = _quantised(h * w) if case["q8"] else (None, None)
        return {"H": H, "Y": Y, "Q": Q, "qscale": rstd * top / 127.0 if case["q8"] else None, "rstd": rstd if case["rstd"] else None}
    if case["op"] == "norm_bwd":
        dY, h, w, rstd = s["dY"].float(), s["H"].float(), s["w"].float(), s["rstd"][:, None]
        n = h * rstd
        g = dY * w
        dH = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if case["dres"]:
            dH = dH + s["dres"].float()
        return {"dH": dH.to(torch.bfloat16), "dw": (dY * n).double().sum(0).float()}
    if case["op"] == "quant":
        Q, top = _quantised(s["A"].float())
        return {"Q": Q, "scale": top / 127.0}
    T, K, N = case["T"], case["K"], case["N"]
    code = _codes(s["meta"])
    place = torch.stack((code & 3, code >> 2), -1).long()
    W = torch.zeros((N, K // 4, 4), device="cuda").scatter_(2, place, s["Wq"].float().view(N, K // 4, 2)).view(N, K)
    Y = (s["Xq"].float() @ W.t()) * s["xs"][:, None] * s["ws"]
    if case["r"]:
        Y = Y + s["XL"].float() @ s["R"].float()
    return {"Y": Y.to(torch.bfloat16)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        H = (s["X"].double() + s["res"].double()).to(torch.bfloat16) if case["res"] else None
        h = (s["X"] if H is None else H).double()
        inv = (h.square().sum(1) / case["D"] + EPS).pow(-0.5)
        y = h * s["w"].double() * inv.unsqueeze(1)
        return {"H": None if H is None else H.double(), "Y": y if case["y"] else None, "Q": None,
                "qscale": y.abs().amax(1) / 127 if case["q8"] else None, "rstd": inv if case["rstd"] else None}
    if case["op"] == "norm_bwd":
        # the Jacobian of n = h rstd applied to g = dY w, with rstd as the forward pass stored it
        dY, h, rstd = s["dY"].double(), s["H"].double(), s["rstd"].double().unsqueeze(1)
        g = dY * s["w"].double()
        dot = (g * h).sum(1, keepdim=True)
        dH = g * rstd - h * (dot * rstd ** 3 / case["D"])
        if case["dres"]:
            dH += s["dres"].double()
        return {"dH": dH, "dw": torch.einsum("td,td->d", dY, h * rstd)}
    if case["op"] == "quant":
        return {"Q": None, "scale": s["A"].double().abs().amax(1) / 127}
    T, K, N = case["T"], case["K"], case["N"]
    X = s["Xq"].double() * s["xs"].double().unsqueeze(1)
    Y = torch.empty((T, N), dtype=torch.float64, device="cuda")
    for n0 in range(0, N, 4096):  # blocks of output channels
        n1 = min(N, n0 + 4096)
        W = torch.zeros((n1 - n0) * K, dtype=torch.float64, device="cuda")
        words = s["meta"][n0:n1].to(torch.int64) & 0xFFFF
        first = torch.arange((n1 - n0) * (K // 16), device="cuda").view(n1 - n0, K // 16) * 16
        v = (s["Wq"][n0:n1].double() * s["ws"][n0:n1].double().unsqueeze(1)).view(n1 - n0, K // 16, 8)
        for j in range(8):  # the kept values of a word, in order
            field = (words >> (2 * j)) & 3
            W[(first + 4 * (j // 2) + field).view(-1)] = v[:, :, j].reshape(-1)
        Y[:, n0:n1] = X @ W.view(n1 - n0, K).t()
    if case["r"]:
        Y += s["XL"].double() @ s["R"].double()
    return {"Y": Y}


def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["D"]
        per = 2 + (4 if case["res"] else 0) + (2 if case["y"] else 0) + (1 if case["q8"] else 0)
        rows = case["T"] * (4 * case["q8"] + 4 * case["rstd"])
        return {"bytes": per * n + rows + 2 * case["D"], "flops": 8 * n}
    if case["op"] == "norm_bwd":
        n = case["T"] * case["D"]
        return {"bytes": (8 if case["dres"] else 6) * n + 4 * case["T"] + 6 * case["D"], "flops": 10 * n}
    if case["op"] == "quant":
        return {"bytes": 3 * case["rows"] * case["K"] + 4 * case["rows"], "flops": 4 * case["rows"] * case["K"]}
    T, K, N, r = case["T"], case["K"], case["N"], case["r"]
    # kept values and codes of the weights, tokens, scales, adapter, output; one multiply-add for each kept weight and token
    return {"bytes": N * K // 2 + N * K // 8 + T * K + 4 * (T + N) + 2 * r * (T + N) + 2 * T * N,
            "flops": T * K * N + 2 * T * r * N}
