"""Bias gradient of the expert layer where a few experts hold nearly all rows, whose sums a whole
cluster shares, beside experts with few rows or none."""
import numpy as np
import pytest
import torch

from oracle import experts
from tests._experts import check, normal, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


CASES = [
    # rows of the experts, N
    ([0, 3000, 1, 700, 0], 264), ([2600, 3, 0, 1, 2500, 0, 0, 2, 7], 8), ([5, 2000], 520), ([2000, 0, 0], 72),
    ([31] * 5 + [5000] + [29] * 10, 264), ([1025, 1024, 1023, 513, 512, 511, 0, 1], 256),
    ([2] * 40 + [9000] + [0] * 22 + [1], 136), ([0] * 1000 + [4500] + [1] * 23, 24), ([600] * 9, 8), ([1, 4097], 1032),
]


@pytest.mark.parametrize("rows,N", CASES)
def test_skewed_shares(rows, N):
    rng = np.random.default_rng(len(rows) + N)
    off, o = offsets_of(rows, 2)
    dY, dYf = normal(rng, (int(o[-1]) + 3, N))
    db = sg.grouped_bias_grad(dY, off)
    depth = np.asarray(rows, dtype=float)[:, None]
    check(db, *experts.grouped_bias_grad(dYf, o), 16 * depth, "db")
    frame = torch.full((len(rows) + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    sg.grouped_bias_grad(dY, off, out=frame[1:-1])
    assert torch.equal(frame[1:-1], db) and (frame[0] == 7.0).all() and (frame[-1] == 7.0).all()


@pytest.mark.parametrize("rows,N", [([0, 3000, 1, 700, 0], 264), ([1500, 3, 0, 1, 2500, 0, 0, 2, 7], 40)])
def test_other_experts_rows_do_not_leak(rows, N):
    rng = np.random.default_rng(3)
    off, o = offsets_of(rows, 1)
    dY, _ = normal(rng, (int(o[-1]) + 1, N))
    clean = sg.grouped_bias_grad(dY, off)
    for e in range(len(rows)):
        bad = dY.clone()
        bad[:int(o[e])] = float("nan")
        bad[int(o[e + 1]):] = float("inf")
        assert torch.equal(sg.grouped_bias_grad(bad, off)[e], clean[e])
