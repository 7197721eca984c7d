"""Plain CPU oracle of the expert (grouped) layer, of microscaled 4-bit and of 8-bit
floating point, in fp64 (test infrastructure only, as the package).

* Expert layer: rows offsets[e] .. offsets[e+1] belong to expert e;
  Y = X W[e]^T + bias[e], dX = dY W[e], dW[e] = dY^T X, dbias[e] = column sums
  of dY over the expert's rows.  Rows of no expert are zero.
* Microscaled 4-bit (OCP Microscaling Formats, MXFP4): a block of 32 along the
  last axis has the scale 2^(floor(log2 max|x|) - 2), the exponent kept in
  -127 .. 127; elements are the nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6} scales,
  ties to the even index of that list, larger ones at 6 scales.  A block that
  holds an infinity or a NaN is NaN.

Every product comes with S, the sum of |term| behind each output element.
"""
from __future__ import annotations

import math

import numpy as np

MX4_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def grouped_forward(X, W, offsets, bias=None):
    """X [T, K], W [E, N, K], bias [E, N], fp64 -> (Y, S) [T, N]."""
    Y = np.zeros((X.shape[0], W.shape[1]))
    S = np.zeros_like(Y)
    for e in range(W.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        Y[r] = X[r] @ W[e].T
        S[r] = np.abs(X[r]) @ np.abs(W[e]).T
        if bias is not None:
            Y[r] += bias[e]
            S[r] += np.abs(bias[e])
    return Y, S


def grouped_backward_input(dY, W, offsets):
    return grouped_forward(dY, np.swapaxes(W, 1, 2), offsets)


def grouped_backward_weight(dY, X, offsets):
    E = len(offsets) - 1
    dW = np.zeros((E, dY.shape[1], X.shape[1]))
    S = np.zeros_like(dW)
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        dW[e] = dY[r].T @ X[r]
        S[e] = np.abs(dY[r]).T @ np.abs(X[r])
    return dW, S


def grouped_bias_grad(dY, offsets):
    parts = [dY[int(a):int(b)] for a, b in zip(offsets, offsets[1:])]
    return np.stack([p.sum(0) for p in parts]), np.stack([np.abs(p).sum(0) for p in parts])


def mx4_block(x):
    """32 numbers -> (4-bit codes, scale byte), plain Python."""
    if any(math.isinf(v) or math.isnan(v) for v in x):
        return [0] * 32, 255
    top = max(abs(v) for v in x)
    e = -127 if top == 0 else max(-127, math.frexp(top)[1] - 1 - 2)
    codes = []
    for v in x:
        m = abs(v) / 2.0 ** e
        dist = [abs(m - level) for level in MX4_LEVELS]
        best = min(dist)
        near = [i for i, d in enumerate(dist) if d == best]
        i = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]
        codes.append(i | (8 if math.copysign(1.0, v) < 0 else 0))
    return codes, e + 127


def mx4_quantize(X):
    """fp64 [R, K] -> codes uint8 [R, K/2] (even column in the low half) and scales uint8 [R, K/32]."""
    R, K = X.shape
    codes = np.zeros((R, K), dtype=np.uint8)
    scales = np.zeros((R, K // 32), dtype=np.uint8)
    for r in range(R):
        for b in range(K // 32):
            c, s = mx4_block([float(v) for v in X[r, 32 * b:32 * b + 32]])
            codes[r, 32 * b:32 * b + 32] = c
            scales[r, b] = s
    return codes[:, 0::2] | codes[:, 1::2] << 4, scales


def mx4_values(codes, scales):
    """Codes and scales -> the fp64 values they stand for."""
    table = np.array(MX4_LEVELS + tuple(-v for v in MX4_LEVELS))
    v = np.empty((*codes.shape[:-1], codes.shape[-1] * 2))
    v[..., 0::2] = table[codes & 15]
    v[..., 1::2] = table[codes >> 4]
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s[scales == 255] = np.nan
    return v * np.repeat(s, 32, axis=-1)


def e4m3_nearest(u):
    """fp64 -> the nearest e4m3 number, ties to the even code, at most 448."""
    m = np.abs(u)
    with np.errstate(divide="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(m > 0, m, 1.0))), -6)   # -6: the subnormal numbers' step is 2^-9
    e = np.where(m >= 2.0 ** (e + 1), e + 1, np.where((m < 2.0 ** e) & (e > -6), e - 1, e))
    step = 2.0 ** (e - 3)
    return np.copysign(np.minimum(np.round(m / step) * step, 448.0), u)


def fp8_quantize(X, block_rows):
    """fp64 (bf16 numbers) [R, K] -> (values of the codes [R, K], scales [rows or tiles, ceil(K / 128)]).

    A block is block_rows x 128; a = max(max|x|, 2^-100), scale a / 448 and factor 448 / a rounded to fp32, the
    product of x and the factor too.  A block that holds an infinity or a NaN has scale NaN and codes 0."""
    R, K = X.shape
    nr, nk = -(-R // block_rows), -(-K // 128)
    codes, scales = np.zeros((R, K)), np.zeros((nr, nk), dtype=np.float32)
    for i in range(nr):
        for j in range(nk):
            at = np.s_[block_rows * i:block_rows * (i + 1), 128 * j:128 * (j + 1)]
            x = X[at]
            if not np.isfinite(x).all():
                scales[i, j] = np.nan
                continue
            a = np.float32(max(np.abs(x).max(), 2.0 ** -100))
            scales[i, j] = a / np.float32(448)
            codes[at] = e4m3_nearest((x.astype(np.float32) * (np.float32(448) / a)).astype(np.float64))
    return codes, scales


def fp8_values(codes, scales):
    """Values of codes [R, K] (as numbers) under scales by row or by tile, fp64."""
    R, K = codes.shape
    s = scales.astype(np.float64)
    s = s if s.shape[0] == R else np.repeat(s, 128, axis=0)[:R]
    return codes * np.repeat(s, 128, axis=1)[:, :K]


def fp8_product(A, As, W, Ws, transposed=False):
    """Rows' code values [T, depth] with scales by row times a weight's [N, K] in tiles (or its transpose):
    (product, S) with S the sum of |term|."""
    a, w = fp8_values(A, As), fp8_values(W, Ws)
    w = w if transposed else w.T
    return a @ w, np.abs(a) @ np.abs(w)


def route(logits, k, score="softmax", renormalize=True, factor=1.0):
    """Logits [T, E], fp64 -> (experts [T, k], weights [T, k], offsets [E + 1], order [T k]), plain Python choices.

    Descending by logit, ties to the lowest expert, NaN after everything; -inf scores 0, in rows of nothing else too."""
    T, E = logits.shape
    experts, weights = np.zeros((T, k), dtype=np.int64), np.zeros((T, k))
    for t in range(T):
        row = [float(v) for v in logits[t]]
        best = sorted(range(E), key=lambda e: (math.isnan(row[e]), -row[e] if not math.isnan(row[e]) else 0.0, e))[:k]
        experts[t] = best
        if score == "softmax":
            top = max(v for v in row) if not any(map(math.isnan, row)) else math.nan
            if top == -math.inf:
                continue
            if math.isnan(top) or top == math.inf:
                weights[t] = math.nan
                continue
            s = np.array([math.exp(row[e] - top) for e in best])
            weights[t] = s / (s.sum() if renormalize else sum(math.exp(v - top) for v in row))
        else:
            s = np.array([math.nan if math.isnan(row[e]) else 0.0 if row[e] < -700 else 1 / (1 + math.exp(-row[e])) for e in best])
            weights[t] = s / (s.sum() or 1.0) if renormalize else s
    flat = experts.ravel()
    order = np.array(sorted(range(T * k), key=lambda p: (flat[p], p)), dtype=np.int64)
    offsets = np.array([int((flat < e).sum()) for e in range(E + 1)])
    return experts, weights * factor, offsets, order


def route_backward(g, logits, experts, score="softmax", renormalize=True, factor=1.0):
    """(gradient of finite logits, S) for the weights' gradient g [T, k]; S the sum of |term|."""
    T, E = logits.shape
    if score == "softmax":
        s = np.exp(logits - logits.max(axis=1, keepdims=True))
        s /= s.sum(axis=1, keepdims=True)
    else:
        s = 1 / (1 + np.exp(-logits))
    grad, S = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        chosen = list(experts[t])
        p = s[t, chosen]
        P = p.sum() if renormalize else 1.0
        # dw_j / ds_i over the choices
        jac = np.eye(len(chosen)) / P - (np.outer(p, np.ones(len(chosen))) / P ** 2 if renormalize else 0.0)
        terms = g[t][:, None] * jac
        ds, dS = np.zeros(E), np.zeros(E)
        ds[chosen], dS[chosen] = terms.sum(0), np.abs(g[t] / P) + (np.abs(g[t] * p).sum() / P ** 2 if renormalize else 0.0)
        if score == "softmax":
            grad[t] = s[t] * (ds - (ds * s[t]).sum())
            S[t] = s[t] * (dS + (dS * s[t]).sum())
        else:
            grad[t] = ds * s[t] * (1 - s[t])
            S[t] = dS * s[t] * (1 - s[t])
    return grad * factor, S * abs(factor)


def moe_forward(X, W13, W2, experts, weights):
    """X [T, H], W13 [E, 2 I, H] (gate, up), W2 [E, H, I], fp64 -> (Y, bound): the layer's output and how far one
    that rounds h to bf16 and sums in fp32 may be from it, before its own rounding.

    Sums of n terms are off by (n / 16 + 8) 2^-22 of their absolute terms (tests/_experts.py); silu has a slope of at
    most 1.1 and its exponential is off by 2^-18 (a fast one, |g| <= 40); the product with the weight by 2^-22 more;
    h is rounded by 2^-8."""
    T, H = X.shape
    I = W2.shape[2]
    Y, B = np.zeros((T, H)), np.zeros((T, H))
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(T):
            for e, w in zip(experts[t], weights[t]):
                if not 0 <= e < W13.shape[0]:
                    continue
                z, S = W13[e] @ X[t], (H / 16 + 8) * 2.0 ** -22 * (np.abs(W13[e]) @ np.abs(X[t]))
                g, u = z[:I], z[I:]
                a = g / (1 + np.exp(-g))
                off = 1.1 * S[:I] * (np.abs(u) + S[I:]) + np.abs(a) * S[I:] + (2.0 ** -18 + 2.0 ** -21) * np.abs(a * u)
                h = w * a * u
                Y[t] += W2[e] @ h
                terms = np.abs(W2[e])
                B[t] += terms @ (2.0 ** -8 * np.abs(h) + (1 + 2.0 ** -8) * abs(w) * off)
                B[t] += (I * len(experts[t]) / 16 + 32) * 2.0 ** -22 * 1.01 * (terms @ (np.abs(h) + abs(w) * off))
    return Y, B
