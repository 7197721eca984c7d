"""Workloads of the expert (grouped) linear layer and of the microscaled 4-bit linear layer.

Expert layer: the rows of X are sorted by expert; rows offsets[e] .. offsets[e+1] are multiplied with
expert e's weight W[e] [N, K].  Rows outside offsets[0] .. offsets[E] belong to no expert and give zeros.
  forward      Y[t] = X[t] W[e]^T + bias[e]
  backward     dX[t] = dY[t] W[e],  dW[e] = sum over e's rows of dY[t]^T X[t],  dbias[e] = sum of dY[t]

4-bit layer (OCP microscaling, MXFP4): 32 neighbours along K share a power-of-two scale
s = 2^(floor(log2 max|x|) - 2) and are rounded to the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6} times s
(ties to even, saturating at 6 s).  Y = Q(X) Q(W)^T + bias, dense or grouped by expert; the weight is
kept in 4 bits, the activations come in bf16.

`own = False` computes the operators in elementary torch operations; `own = True` calls the library.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one token routed to two of eight experts
        dict(name="experts_token", op="fwd", T=2, E=8, K=2048, N=4096, idle=0, spare=0, skew=0.0, bias=False),
        # a decoding batch: a few rows for each of sixteen experts, MLP of the decode workload
        dict(name="experts_decode", op="fwd", T=64, E=16, K=4096, N=11008, idle=0, spare=0, skew=0.7, bias=False),
        # odd sizes, experts without a row, padding rows behind the last expert's
        dict(name="experts_ragged", op="fwd", T=1531, E=11, K=1000, N=712, idle=3, spare=37, skew=1.0, bias=True),
        # a long prompt through an MLP projection of the large workload's size
        dict(name="experts_prefill", op="fwd", T=16384, E=8, K=4096, N=14336, idle=0, spare=0, skew=0.4, bias=False),
        # a small training step with odd sizes, an idle expert and padding rows
        dict(name="experts_train_ragged", op="bwd", T=777, E=5, K=776, N=1032, idle=1, spare=9, skew=0.8, bias=True),
        # gradients of a training step at the large workload's size
        dict(name="experts_train", op="bwd", T=8192, E=8, K=4096, N=14336, idle=0, spare=0, skew=0.4, bias=True),
        # activations of a small batch to 4 bits and back
        dict(name="mx4_tokens", op="quant", T=33, K=4096),
        # a layer's weight to 4 bits and back
        dict(name="mx4_weight", op="quant", T=14336, K=4096),
        # one token through a 4-bit layer
        dict(name="mx4_token", op="mx4", T=1, K=4096, N=11008, bias=True),
        # a long prompt through a 4-bit layer
        dict(name="mx4_prefill", op="mx4", T=8192, K=4096, N=14336, bias=False),
        # a decoding batch through 4-bit experts
        dict(name="mx4_experts_decode", op="gmx4", T=64, E=16, K=4096, N=11008, idle=0, spare=0, skew=0.7,
             bias=False),
        # a long prompt through 4-bit experts
        dict(name="mx4_experts_prefill", op="gmx4", T=16384, E=8, K=4096, N=14336, idle=0, spare=0, skew=0.4,
             bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, m):
    return max(lo, _log_int(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "quant", "mx4", "gmx4", "gmx4"])
    if op == "quant":
        return dict(op=op, T=_log_int(rng, 1, 14336), K=_multiple(rng, 32, 4096, 32))
    step = 32 if op in ("mx4", "gmx4") else 8
    case = dict(op=op, K=_multiple(rng, 256, 4096, step), N=_multiple(rng, 256, 11008, 8), bias=rng.random() < 0.5)
    if op == "mx4":
        case["T"] = _log_int(rng, 1, 8192)
        return case
    case["E"] = _log_int(rng, 1, 16)
    case["T"] = _log_int(rng, 1, 8192)
    case["idle"] = rng.randrange(0, max(1, case["E"] // 2))
    case["spare"] = rng.choice([0, 0, rng.randrange(0, 64)])
    case["skew"] = rng.choice([0.0, 0.4, 0.8, 1.2])
    return case


# ---------------------------------------------------------------- inputs


def _rows(case):
    """Rows of the experts (descending): T rows over E - idle experts, shares (i + 1)^-skew."""
    live = max(1, case["E"] - case["idle"])
    w = [(i + 1) ** -case["skew"] for i in range(live)]
    cut = [0]
    for i in range(live):
        cut.append(round(case["T"] * sum(w[: i + 1]) / sum(w)))
    rows = [b - a for a, b in zip(cut, cut[1:])]
    if case["T"] <= live:  # fewer rows than experts: one each
        rows = [1] * case["T"] + [0] * (live - case["T"])
    return rows + [0] * (case["E"] - live)


def _normal(gen, shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for part in (out if out.dim() == 3 else [out]):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * std)
    return out


def _tokens(gen, T, K):
    """Activations: normal rows of differing scale with a few outlying channels."""
    x = torch.randn((T, K), generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=gen, device=DEV))
    x *= 1.0 + 7.0 * (torch.rand((1, K), generator=gen, device=DEV) < 0.01)
    return x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, T, K = case["op"], case["T"], case["K"]
    s = {"op": op}
    if op == "quant":
        s["X"] = _tokens(gen, T, K)
        return s
    N = case["N"]
    if op == "mx4":
        s["X"] = _tokens(gen, T, K)
        W = _normal(gen, (1, N, K), K ** -0.5)
        bias_shape = (N,)
    else:
        E = case["E"]
        rows = _rows(case)
        order = torch.randperm(E, generator=gen, device=DEV).tolist()
        ends = [0]
        for e in order:
            ends.append(ends[-1] + rows[e])
        s["ends"] = ends
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        total = T + case["spare"]
        s["X"] = _tokens(gen, total, K) if op == "gmx4" else _normal(gen, (total, K))
        W = _normal(gen, (E, N, K), K ** -0.5)
        bias_shape = (E, N)
        if op == "bwd":
            s["dY"] = _normal(gen, (total, N), 0.01)
    s["bias"] = _normal(gen, bias_shape) if case["bias"] else None
    if op in ("fwd", "bwd"):
        s["W"] = W
        if own:
            import sparse_gemm_b200 as sg
            s["handle"] = sg.GroupedWeight(W)
        return s
    # 4-bit weights: two codes a byte, the even column in the low half, and one scale code for 32 columns
    codes = torch.empty((*W.shape[:2], K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((*W.shape[:2], K // 32), dtype=torch.uint8, device=DEV)
    for e in range(W.shape[0]):
        for r in range(0, N, 2048):
            c, x = _encode(W[e, r:r + 2048].float())
            codes[e, r:r + 2048] = c[:, 0::2] | (c[:, 1::2] << 4)
            scales[e, r:r + 2048] = (x + 127).to(torch.uint8)
    if op == "mx4":
        codes, scales = codes[0], scales[0]
    s["codes"], s["scales"] = codes, scales
    if own:
        import sparse_gemm_b200 as sg
        s["handle"] = sg.Mx4Tensor(codes, scales)
    return s


# ---------------------------------------------------------------- plain form


def _pow2(e):
    """2^e in 64 bits, from the number's exponent field (e in the normal range)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _encode(x):
    """fp32 [R, K] (finite) -> 4-bit codes [R, K] (sign in bit 3) and scale exponents [R, K / 32]."""
    blocks = x.reshape(x.shape[0], -1, 32)
    top = blocks.abs().amax(dim=2)
    # floor(log2 top) is the exponent field of the fp32 number (0 below the normal range: clamped below)
    exponent = ((top.view(torch.int32) >> 23) - 127).clamp(-125, 127) - 2
    mag = (blocks.abs().double() * _pow2(-exponent)[:, :, None]).float()
    # halfway points between 0, .5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code
    code = (mag > 0.25).to(torch.uint8)
    for border, inclusive in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (mag >= border) if inclusive else (mag > border)
    sign = torch.signbit(blocks).to(torch.uint8) << 3
    return (code | sign).reshape(x.shape), exponent


def _level(code):
    """Values of 4-bit codes, fp32."""
    c = (code & 7).float()
    mag = torch.where(c < 4, c * 0.5, torch.where(c < 6, c - 2.0, 2.0 * c - 8.0))
    return torch.where(code >= 8, -mag, mag)


def _scaled(code, exponent):
    """Values of codes [R, K] under scale exponents [R, K / 32], fp32."""
    v = _level(code).reshape(code.shape[0], -1, 32)
    return (v.double() * _pow2(exponent)[:, :, None]).float().reshape(code.shape)


def _unpack(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1)
    return _scaled(c, scales.to(torch.int32) - 127)


def _affine(y, bias):
    return (y if bias is None else y + bias.float()).to(torch.bfloat16)


def _plain(s):
    op, X = s["op"], s["X"]
    if op == "quant":
        return _scaled(*_encode(X.float())).to(torch.bfloat16)
    if op == "mx4":
        return _affine(_scaled(*_encode(X.float())) @ _unpack(s["codes"], s["scales"]).T, s["bias"])
    ends = s["ends"]
    if op == "bwd":
        W, dY = s["W"], s["dY"]
        dX, dW = torch.zeros_like(X), torch.zeros_like(W)
        db = torch.zeros(W.shape[:2], dtype=torch.bfloat16, device=X.device)
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if b > a:
                g = dY[a:b].float()
                dX[a:b] = (g @ W[e].float()).to(torch.bfloat16)
                dW[e] = (g.T @ X[a:b].float()).to(torch.bfloat16)
                db[e] = g.sum(dim=0).to(torch.bfloat16)
        return dX, dW, db
    N = s["codes"].shape[1] if op == "gmx4" else s["W"].shape[1]
    Y = torch.zeros((X.shape[0], N), dtype=torch.bfloat16, device=X.device)
    x = _scaled(*_encode(X.float())) if op == "gmx4" else X.float()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if b > a:
            w = _unpack(s["codes"][e], s["scales"][e]) if op == "gmx4" else s["W"][e].float()
            Y[a:b] = _affine(x[a:b] @ w.T, None if s["bias"] is None else s["bias"][e])
    return Y


def run(state):
    if not own:
        return _plain(state)
    import sparse_gemm_b200 as sg
    s = state
    if s["op"] == "quant":
        return sg.dequantize_mx4(sg.quantize_mx4(s["X"]))
    if s["op"] == "mx4":
        return sg.forward_mx4(s["X"], s["handle"], bias=s["bias"])
    if s["op"] == "gmx4":
        return sg.grouped_forward_mx4(s["X"], s["handle"], s["offsets"], bias=s["bias"])
    if s["op"] == "fwd":
        return sg.grouped_forward(s["X"], s["handle"], s["offsets"], bias=s["bias"])
    return (sg.grouped_backward_input(s["dY"], s["handle"], s["offsets"]),
            sg.grouped_backward_weight(s["dY"], s["X"], s["handle"], s["offsets"]),
            sg.grouped_bias_grad(s["dY"], s["offsets"]))


# ---------------------------------------------------------------- work


def work(case):
    op, T, K = case["op"], case["T"], case["K"]
    if op == "quant":
        return {"bytes": 4 * T * K, "flops": 2 * T * K}
    N = case["N"]
    if op == "mx4":
        live, total, E = 1, T, 1
    else:
        live = sum(r > 0 for r in _rows(case))
        total, E = T + case["spare"], case["E"]
    bias = 2 * live * N if case["bias"] else 0
    if op == "bwd":
        return {"bytes": 2 * (T * N + T * K + live * N * K + total * K + E * N * K + E * N),
                "flops": 4 * T * N * K + T * N}
    weight = live * N * K * (2 if op == "fwd" else 17 / 32)
    return {"bytes": int(2 * T * K + weight + bias + 2 * total * N), "flops": 2 * T * N * K}


# ---------------------------------------------------------------- definition in 64 bits


def _powers(device):
    """2^-127 .. 2^127."""
    return torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=torch.float64, device=device)


def _nearest(x):
    """The 4-bit layer's rounding of bf16 [R, K], from the definition, in 64 bits."""
    v = x.double().reshape(x.shape[0], -1, 32)
    powers = _powers(x.device)
    top = v.abs().amax(dim=2, keepdim=True)
    # largest i in -127 .. 127 with 2^(i + 2) <= top, else -127
    e = (torch.bucketize(top, powers * 4, right=True) - 1).clamp(min=0)
    u = (v.abs() / powers[e]).clamp(max=6.0)
    # spacing of the levels at u: .5 below 2, 1 below 4, else 2; round() takes ties to even multiples
    step = torch.where(u < 2, 0.5, torch.where(u < 4, 1.0, 2.0))
    q = torch.round(u / step) * step
    return (torch.copysign(q, v) * powers[e]).reshape(x.shape)


def _decode(codes, scales):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device=codes.device)
    v = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    v[:, 0::2] = table[(codes % 16).long()]
    v[:, 1::2] = table[(codes // 16).long()]
    return v * _powers(codes.device)[scales.long()].repeat_interleave(32, dim=1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, X = case["op"], s["X"]
    if op == "quant":
        return _nearest(X)
    bias = s["bias"]
    if op == "mx4":
        Y = torch.matmul(_nearest(X), _decode(s["codes"], s["scales"]).t())
        return Y if bias is None else Y.add_(bias.double())
    o = s["offsets"].cpu()
    spans = [(e, slice(int(o[e]), int(o[e + 1]))) for e in range(case["E"])]
    if op == "bwd":
        dX = torch.zeros(X.shape, dtype=torch.float64, device=DEV)
        dW = torch.zeros(s["W"].shape, dtype=torch.float64, device=DEV)
        db = torch.zeros((case["E"], case["N"]), dtype=torch.float64, device=DEV)
        for e, r in spans:
            g = s["dY"][r].double()
            dX[r] = torch.matmul(g, s["W"][e].double())
            dW[e] = torch.matmul(g.t(), X[r].double())
            db[e] = g.sum(0)
        return dX, dW, db
    Y = torch.zeros((X.shape[0], case["N"]), dtype=torch.float64, device=DEV)
    for e, r in spans:
        if r.start == r.stop:
            continue
        if op == "gmx4":
            Y[r] = torch.matmul(_nearest(X[r]), _decode(s["codes"][e], s["scales"][e]).t())
        else:
            Y[r] = torch.matmul(X[r].double(), s["W"][e].double().t())
        if bias is not None:
            Y[r] += bias[e].double()
    return Y
