"""Plain CPU oracle of the expert (grouped) layer and of microscaled 4-bit
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
