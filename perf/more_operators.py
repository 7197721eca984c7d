"""Workloads of the 8-bit layer with a scale for each block of 128, of the experts' router, and of a whole
mixture-of-experts layer for a few tokens.

8-bit layer (e4m3, values up to 448): an activation row shares a scale among 128 neighbours along K, a weight
among tiles of 128 x 128 (the last of a row or column may be shorter).  With a = max(max|x|, 2^-100) over a block,
rounded to fp32 where a step is named:
  scale s = a / 448 (fp32),  r = 448 / a (fp32),  code = e4m3(x r (fp32)), to nearest, ties to even
The value of a code is code times s.  Products of codes and scales, dense or grouped by expert (rows
offsets[e] .. offsets[e+1] of X belong to expert e, rows of no expert give zeros):
  forward          Y[t] = Q(X)[t] Q(W[e])^T + bias[e]
  input gradient   dX[t] = Q(dY)[t] Q(W[e])

Router: from logits [T, E] the k largest of each row (ties to the lowest expert), their scores
  softmax: s_i = exp(l_i) / sum_j exp(l_j)     sigmoid: s_i = 1 / (1 + exp(-l_i))
as weights (renormalised to a sum of one where asked for, times a factor), the pairs (token, choice) sorted by
expert, and the gradient of the logits.

Mixture-of-experts layer for a few tokens: with e_j, w_j a token's experts and weights, and W13[e] = (gate, up),
  y = sum_j w_j W2[e_j] (silu(gate[e_j] x) * (up[e_j] x))
with bf16 weights, or 8-bit ones as above (the activations stay as they are).

`own = False` computes the operators in elementary torch operations; `own = True` calls the library.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # activations of a small batch to 8 bits and back, odd sizes
        dict(name="fp8_tokens", op="quant", rows=1, T=37, K=4016),
        # a layer's weight to 8 bits and back
        dict(name="fp8_weight", op="quant", rows=128, T=14336, K=4096),
        # one token through an 8-bit layer, MLP of the decode workload
        dict(name="fp8_token", op="fp8", T=1, K=4096, N=11008, bias=True),
        # a long prompt through an MLP projection of the large workload's size
        dict(name="fp8_prefill", op="fp8", T=8192, K=4096, N=14336, bias=False),
        # a decoding batch: a few rows for each of sixteen experts
        dict(name="fp8_experts_decode", op="gfp8", T=64, E=16, K=4096, N=11008, idle=0, spare=0, skew=0.7, bias=False),
        # odd sizes, experts without a row, padding rows behind the last expert's, both directions
        dict(name="fp8_experts_ragged", op="both", T=1531, E=11, K=1008, N=720, idle=3, spare=37, skew=1.0, bias=True),
        # the gradient that a training step sends back through experts of the large workload's size
        dict(name="fp8_experts_grad", op="grad", T=8192, E=8, K=4096, N=14336, idle=0, spare=0, skew=0.4),
        # a decoding batch's router in half precision, with equal logits in many rows
        dict(name="route_tokens", op="route", T=61, E=64, k=6, score="sigmoid", renorm=True, half=True),
        # the router of a long prompt in training, forward and backward
        dict(name="route_train", op="route", T=16384, E=128, k=8, score="softmax", renorm=False, half=False),
        # one token through a whole expert layer of the large workload's size
        dict(name="moe_token", op="moe", T=1, E=8, k=2, H=4096, I=14336, fp8=False, skew=0.0),
        # a few tokens through a small layer of odd sizes
        dict(name="moe_ragged", op="moe", T=13, E=11, k=3, H=1000, I=712, fp8=False, skew=1.0),
        # a decoding batch through many small experts in 8 bits
        dict(name="moe_batch", op="moe", T=32, E=64, k=6, H=2048, I=1408, fp8=True, skew=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, m):
    return max(lo, _log_int(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["quant", "fp8", "gfp8", "both", "grad", "route", "moe", "moe"])
    if op == "quant":
        return dict(op=op, rows=rng.choice([1, 128]), T=_log_int(rng, 1, 14336), K=_multiple(rng, 32, 4096, 16))
    if op == "route":
        E = _log_int(rng, 2, 256)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E)),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5, half=rng.random() < 0.3)
    if op == "moe":
        fp8 = rng.random() < 0.5
        E = _log_int(rng, 2, 64)
        return dict(op=op, T=_log_int(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)),
                    H=_multiple(rng, 256, 4096, 16 if fp8 else 8),
                    I=_multiple(rng, 256, 14336 if E <= 8 else 2048, 16 if fp8 else 8), fp8=fp8,
                    skew=rng.choice([0.0, 0.5, 1.0]))
    case = dict(op=op, K=_multiple(rng, 256, 4096, 16), N=_multiple(rng, 256, 11008, 8 if op in ("fp8", "gfp8") else 16),
                T=_log_int(rng, 1, 8192))
    if op != "grad":
        case["bias"] = rng.random() < 0.5
    if op != "fp8":
        case["E"] = _log_int(rng, 1, 16)
        case["idle"] = rng.randrange(0, max(1, case["E"] // 2))
        case["spare"] = rng.choice([0, 0, rng.randrange(0, 64)])
        case["skew"] = rng.choice([0.0, 0.4, 0.8, 1.2])
    return case


# ---------------------------------------------------------------- inputs


def _rows(case):
    """Rows of the experts (descending): T rows over E - idle experts, shares (i + 1)^-skew."""
    live = max(1, case["E"] - case["idle"])
    if case["T"] <= live:  # fewer rows than experts: one each
        return [1] * case["T"] + [0] * (case["E"] - case["T"])
    w = [(i + 1) ** -case["skew"] for i in range(live)]
    cut = [0]
    for i in range(live):
        cut.append(round(case["T"] * sum(w[: i + 1]) / sum(w)))
    return [b - a for a, b in zip(cut, cut[1:])] + [0] * (case["E"] - live)


def _normal(gen, shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for part in (out if out.dim() == 3 else [out]):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * std)
    return out


def _tokens(gen, T, K, std=1.0):
    """Activations: normal rows of differing scale with a few outlying channels."""
    x = torch.randn((T, K), generator=gen, device=DEV) * std
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=gen, device=DEV))
    x *= 1.0 + 7.0 * (torch.rand((1, K), generator=gen, device=DEV) < 0.01)
    return x.to(torch.bfloat16)


def _weight8(gen, E, N, K):
    """Experts' weights in 8 bits: codes [E, N, K] and the scales of their tiles."""
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((E, -(-N // 128), -(-K // 128)), dtype=torch.float32, device=DEV)
    for e in range(E):
        w = (torch.randn((N, K), generator=gen, device=DEV) * K ** -0.5).to(torch.bfloat16)
        codes[e], scales[e] = _encode(w, 128)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, T = case["op"], case["T"]
    s = dict(case)
    if own:
        import sparse_gemm_b200 as sg
    if op == "quant":
        s["X"] = _tokens(gen, T, case["K"])
        return s
    if op in ("route", "moe"):
        E, k = case["E"], case["k"]
        logits = torch.randn((T, E), generator=gen, device=DEV) * 1.5
        # some experts are liked more than others
        logits += case.get("skew", 0.5) * torch.randn((1, E), generator=gen, device=DEV)
        s["logits"] = logits.to(torch.bfloat16) if case.get("half") else logits
        if op == "route":
            s["g"] = torch.randn((T, k), generator=gen, device=DEV)
            return s
        H, I = case["H"], case["I"]
        s["X"] = _tokens(gen, T, H)
        if case["fp8"]:
            s["W13"], s["W2"] = _weight8(gen, E, 2 * I, H), _weight8(gen, E, H, I)
        else:
            s["W13"], s["W2"] = _normal(gen, (E, 2 * I, H), H ** -0.5), _normal(gen, (E, H, I), I ** -0.5)
        if own:
            s["h13"], s["h2"] = ((sg.Fp8Tensor(*s[w]) if case["fp8"] else sg.GroupedWeight(s[w])) for w in ("W13", "W2"))
        return s
    K, N, E = case["K"], case["N"], case.get("E", 1)
    total = T
    if op != "fp8":
        rows = _rows(case)
        order = torch.randperm(E, generator=gen, device=DEV).tolist()
        ends = [0]
        for e in order:
            ends.append(ends[-1] + rows[e])
        s["ends"] = ends
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        total += case["spare"]
    if op != "grad":
        s["X"] = _tokens(gen, total, K)
    if op in ("both", "grad"):
        s["dY"] = _tokens(gen, total, N, 0.01)
    s["bias"] = _normal(gen, (N,) if op == "fp8" else (E, N)) if case.get("bias") else None
    codes, scales = _weight8(gen, E, N, K)
    s["codes"], s["scales"] = (codes[0], scales[0]) if op == "fp8" else (codes, scales)
    if own:
        s["handle"] = sg.Fp8Tensor(s["codes"], s["scales"])
    return s


# ---------------------------------------------------------------- plain form


def _blocks(x, rows):
    """[R, K] padded with zeros to [blocks of rows, rows, blocks of 128, 128]."""
    R, K = x.shape
    padded = torch.zeros((-(-R // rows) * rows, -(-K // 128) * 128), dtype=x.dtype, device=x.device)
    padded[:R, :K] = x
    return padded.view(-1, rows, padded.shape[1] // 128, 128)


def _encode(x, rows):
    """bf16 [R, K] -> codes and scales of blocks of `rows` x 128."""
    v = _blocks(x.float(), rows)
    a = v.abs().amax(dim=(1, 3)).clamp(min=2.0 ** -100)
    r = 448.0 / a
    codes = (v * r[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.reshape(-1, v.shape[2] * 128)[: x.shape[0], : x.shape[1]].contiguous(), a / 448.0


def _decode(codes, scales):
    """Values of codes [R, K], fp32; scales of one row or of tiles."""
    R, K = codes.shape
    s = scales if scales.shape[0] == R else scales.repeat_interleave(128, dim=0)[:R]
    return codes.float() * s.repeat_interleave(128, dim=1)[:, :K]


def _affine(y, bias):
    return (y if bias is None else y + bias.float()).to(torch.bfloat16)


def _plain_route(s):
    logits = s["logits"].float()
    T, E, k = logits.shape[0], logits.shape[1], s["k"]
    experts = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    score = torch.softmax(logits, dim=1) if s.get("score", "softmax") == "softmax" else torch.sigmoid(logits)
    chosen = torch.gather(score, 1, experts)
    total = chosen.sum(dim=1, keepdim=True) if s.get("renorm", True) else 1.0
    weights = chosen / total
    if s["op"] == "moe":
        return experts.int(), weights
    flat = experts.flatten()
    order = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=logits.device)
    offsets[1:] = torch.cumsum((flat[:, None] == torch.arange(E, device=flat.device)).sum(dim=0), dim=0)
    # gradient: of the chosen scores, then of the logits
    g = s["g"]
    if s["renorm"]:
        g = (g - (g * weights).sum(dim=1, keepdim=True)) / total
    ds = torch.zeros_like(score).scatter(1, experts, g)
    if s["score"] == "softmax":
        grad = score * (ds - (ds * score).sum(dim=1, keepdim=True))
    else:
        grad = ds * score * (1 - score)
    return experts.int(), weights, offsets, order.int(), grad.to(s["logits"].dtype)


def _plain_moe(s):
    experts, weights = _plain_route(s)
    X = s["X"].float()
    Y = torch.zeros_like(X)
    for e in torch.unique(experts).tolist():
        t, j = torch.nonzero(experts == e, as_tuple=True)
        W13, W2 = ((_decode(w[0][e], w[1][e]) if s["fp8"] else w[e].float()) for w in (s["W13"], s["W2"]))
        gate, up = (X[t] @ W13.T).chunk(2, dim=1)
        Y.index_add_(0, t, weights[t, j, None] * ((gate / (1 + torch.exp(-gate)) * up) @ W2.T))
    return Y.to(torch.bfloat16)


def _plain(s):
    op = s["op"]
    if op == "quant":
        codes, scales = _encode(s["X"], s["rows"])
        return _decode(codes, scales).to(torch.bfloat16), scales
    if op == "route":
        return _plain_route(s)
    if op == "moe":
        return _plain_moe(s)
    if op == "fp8":
        return _affine(_decode(*_encode(s["X"], 1)) @ _decode(s["codes"], s["scales"]).T, s["bias"])
    N, K = s["codes"].shape[1:]
    out = []
    for name, width in (("X", N), ("dY", K)):
        if name not in s:
            continue
        x = _decode(*_encode(s[name], 1))
        y = torch.zeros((x.shape[0], width), dtype=torch.bfloat16, device=x.device)
        for e, (a, b) in enumerate(zip(s["ends"], s["ends"][1:])):
            if b > a:
                w = _decode(s["codes"][e], s["scales"][e])
                if name == "X":
                    y[a:b] = _affine(x[a:b] @ w.T, None if s["bias"] is None else s["bias"][e])
                else:
                    y[a:b] = (x[a:b] @ w).to(torch.bfloat16)
        out.append(y)
    return out


def run(state):
    if not own:
        return _plain(state)
    import sparse_gemm_b200 as sg
    s, op = state, state["op"]
    if op == "quant":
        q = sg.quantize_fp8(s["X"], block_rows=s["rows"])
        return sg.dequantize_fp8(q), q.scales
    if op == "route":
        r = sg.route(s["logits"], s["k"], score=s["score"], renormalize=s["renorm"])
        return (r.experts, r.weights, r.offsets, r.order,
                sg.route_backward(s["g"], s["logits"], r.experts, score=s["score"], renormalize=s["renorm"]))
    if op == "moe":
        r = sg.route(s["logits"], s["k"], sort=False)
        return sg.moe_forward(s["X"], s["h13"], s["h2"], r.experts, r.weights)
    if op == "fp8":
        return sg.forward_fp8(s["X"], s["handle"], bias=s["bias"])
    out = []
    if "X" in s:
        out.append(sg.grouped_forward_fp8(s["X"], s["handle"], s["offsets"], bias=s["bias"]))
    if "dY" in s:
        out.append(sg.grouped_backward_input_fp8(s["dY"], s["handle"], s["offsets"]))
    return out


# ---------------------------------------------------------------- work


def _tiles(N, K):
    return -(-N // 128) * -(-K // 128)


def work(case):
    op, T = case["op"], case["T"]
    if op == "quant":
        K = case["K"]
        return {"bytes": 4 * T * K + 4 * _tiles(T * 128 // case["rows"], K), "flops": 2 * T * K}
    if op == "route":
        E, k = case["E"], case["k"]
        size = 2 if case["half"] else 4
        return {"bytes": 2 * T * E * size + 16 * T * k + 4 * E + 4, "flops": 6 * T * E}
    if op == "moe":
        H, I, pairs = case["H"], case["I"], T * case["k"]
        # the experts that independent choices reach, as an expectation
        live = max(case["k"], round(case["E"] * (1 - (1 - case["k"] / case["E"]) ** T)))
        weight = 3 * H * I + 4 * (_tiles(2 * I, H) + _tiles(H, I)) if case["fp8"] else 6 * H * I
        return {"bytes": live * weight + 4 * T * H + 4 * T * case["E"], "flops": 6 * pairs * H * I}
    K, N = case["K"], case["N"]
    live, total = 1, T
    if op != "fp8":
        live, total = sum(r > 0 for r in _rows(case)), T + case["spare"]
    weight = live * (N * K + 4 * _tiles(N, K))
    bias = 2 * live * N if case.get("bias") else 0
    forward = 2 * T * K + weight + bias + 2 * total * N
    grad = 2 * T * N + weight + 2 * total * K
    return {"bytes": grad if op == "grad" else forward + (grad if op == "both" else 0),
            "flops": 2 * T * N * K * (2 if op == "both" else 1)}


# ---------------------------------------------------------------- definition in 64 bits


def _nearest8(u):
    """The nearest e4m3 number of u (64 bits), ties to even: three bits behind the leading one, steps of 2^-9 below."""
    m, e = torch.frexp(u)
    step = torch.ldexp(torch.ones_like(u), (e - 4).clamp(min=-9))
    return (torch.round(u / step) * step).clamp(-448.0, 448.0)


def _rounded8(x, rows):
    """Values that bf16 [R, K] becomes in 8 bits, and the scales, block by block of the columns."""
    R, K = x.shape
    out = torch.empty((R, K), dtype=torch.float64, device=x.device)
    scales = []
    for c in range(0, K, 128):
        v = x[:, c:c + 128].double()
        top = v.abs().amax(dim=1)
        if rows > 1:
            pad = torch.zeros(-(-R // rows) * rows, dtype=torch.float64, device=x.device)
            pad[:R] = top
            top = pad.view(-1, rows).amax(dim=1)
        top = torch.maximum(top, torch.full_like(top, 2.0 ** -100))
        s = (top / 448.0).float().double()
        r = (448.0 / top).float().double()
        scales.append(s)
        if rows > 1:
            s, r = (w.repeat_interleave(rows)[:R] for w in (s, r))
        out[:, c:c + 128] = _nearest8((v * r[:, None]).float().double()) * s[:, None]
    return out, torch.stack(scales, dim=1)


def _stored8(codes, scales):
    """Values of an expert's stored weight, tile by tile."""
    v = codes.double()
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            v[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= scales[i, j].double()
    return v


def _exact_route(s):
    l = s["logits"].double()
    T, E, k = l.shape[0], l.shape[1], s["k"]
    idx = torch.arange(E, device=l.device)
    experts = torch.empty((T, k), dtype=torch.int64, device=l.device)
    for a in range(0, T, 1024):
        x = l[a:a + 1024]
        ahead = (x[:, None, :] > x[:, :, None]) | ((x[:, None, :] == x[:, :, None]) & (idx[None, :] < idx[:, None]))
        rank = ahead.sum(dim=2)
        for j in range(k):
            experts[a:a + 1024, j] = (rank == j).to(torch.int8).argmax(dim=1)
    if s.get("score", "softmax") == "softmax":
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    w = torch.take_along_dim(p, experts, dim=1)
    if s.get("renorm", True):
        w = w / w.sum(dim=1, keepdim=True)
    return p, experts, w


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "quant":
        return _rounded8(s["X"], case["rows"])
    if op == "route":
        p, experts, w = _exact_route(s)
        T, k, E = case["T"], case["k"], case["E"]
        flat = experts.flatten()
        order = torch.cat([torch.nonzero(flat == e).flatten() for e in range(E)])
        offsets = torch.searchsorted(flat[order].contiguous(), torch.arange(E + 1, device=DEV))
        g = s["g"].double()
        picked = torch.take_along_dim(p, experts, dim=1)
        if case["renorm"]:  # w_j = p_j / P: dp_j = g_j / P - sum_i g_i p_i / P^2
            P = picked.sum(dim=1, keepdim=True)
            g = g / P - (g * picked).sum(dim=1, keepdim=True) / P ** 2
        grad = torch.zeros_like(p)
        if case["score"] == "sigmoid":
            grad.scatter_(1, experts, g * picked * (1 - picked))
        else:  # dl_i = sum_j g_j p_j (delta_ij - p_i)
            grad -= p * (g * picked).sum(dim=1, keepdim=True)
            grad.scatter_add_(1, experts, g * picked)
        return experts.int(), w, offsets.int(), order.int(), grad
    if op == "moe":
        _, experts, w = _exact_route(s)
        X = s["X"].double()
        Y = torch.zeros_like(X)
        I = case["I"]
        for e in range(case["E"]):
            share = (w * (experts == e)).sum(dim=1)
            t = torch.nonzero((experts == e).any(dim=1)).flatten()
            if not len(t):
                continue
            W13, W2 = ((_stored8(m[0][e], m[1][e]) if case["fp8"] else m[e].double()) for m in (s["W13"], s["W2"]))
            gate, up = torch.matmul(X[t], W13[:I].t()), torch.matmul(X[t], W13[I:].t())
            Y[t] += share[t, None] * torch.matmul(gate * torch.sigmoid(gate) * up, W2.t())
        return Y
    if op == "fp8":
        Y = torch.matmul(_rounded8(s["X"], 1)[0], _stored8(s["codes"], s["scales"]).t())
        return Y if s["bias"] is None else Y.add_(s["bias"].double())
    o = s["offsets"].cpu()
    spans = [(e, slice(int(o[e]), int(o[e + 1]))) for e in range(case["E"])]
    out = []
    for name, width in (("X", case["N"]), ("dY", case["K"])):
        if name not in s:
            continue
        Y = torch.zeros((s[name].shape[0], width), dtype=torch.float64, device=DEV)
        for e, r in spans:
            if r.start == r.stop:
                continue
            W = _stored8(s["codes"][e], s["scales"][e])
            Y[r] = torch.matmul(_rounded8(s[name][r], 1)[0], W.t() if name == "X" else W)
            if name == "X" and s["bias"] is not None:
                Y[r] += s["bias"][e].double()
        out.append(Y)
    return out
