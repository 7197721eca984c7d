"""Inputs and bounds shared by the GPU tests of the expert layer and the 4-bit layer.

Bound.  Outputs are fp32 sums y' rounded once to bf16 (half a step: 2^-8 of the
value).  The tensor cores add 16 or more products to the accumulator at a time,
each addition off by at most 2^-22 of the sum of |terms| S (one fp32 step,
doubled for truncation), so with ceil(depth / 16) additions, 8 more for the
bias and partial sums,
    |y - ref| <= 2^-8 |ref| + (1 + 2^-8) (ceil(depth / 16) + 8) 2^-22 S.
"""
import numpy as np
import torch

import synth
from tests._gpu import to_dev


def check(got: torch.Tensor, ref: np.ndarray, S: np.ndarray, depth, what=""):
    got = got.detach().float().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (np.ceil(depth / 16) + 8) * 2.0 ** -22 * S
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first {i}: got {got[i]!r}, "
                             f"ref {ref[i]!r}, bound {bound[i]!r}")


def normal(rng, shape, std=1.0):
    """bf16 normals as (CUDA tensor, fp64 array)."""
    b = synth.bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))
    return to_dev(b), synth.bits_to_f32(b).astype(np.float64)


def integers(rng, shape, lo=-3, hi=3):
    b = synth.bf16_bits(rng.integers(lo, hi + 1, shape).astype(np.float32))
    return to_dev(b), synth.bits_to_f32(b).astype(np.float64)


def offsets_of(rows, first=0):
    o = np.concatenate([[first], first + np.cumsum(rows)]).astype(np.int32)
    return torch.from_numpy(o).cuda(), o
