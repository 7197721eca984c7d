"""Weight gradient over every number of rows up to two stages: an expert's last rows come in copies of
their own, with zeros behind them, whatever the neighbours' rows hold."""
import numpy as np
import pytest
import torch

from oracle import experts
from tests._experts import integers, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


@pytest.mark.parametrize("N,K", [(72, 136), (264, 64), (8, 328)])
@pytest.mark.parametrize("junk", [0.0, float("nan"), float("inf")])
def test_every_number_of_rows(N, K, junk):
    """Experts of 1 .. 257 rows in turn with experts whose rows are NaN, infinite or zero: sums of small
    integers are exact, and nothing of a neighbour's row reaches them."""
    rng = np.random.default_rng(91)
    rows = [r for n in range(1, 258) for r in (n, 3)] + [3]
    off, o = offsets_of(rows, 5)
    T = int(o[-1]) + 1
    (X, Xf), (dY, dYf) = integers(rng, (T, K)), integers(rng, (T, N))
    Wg = sg.GroupedWeight(torch.zeros(len(rows), N, K, dtype=torch.bfloat16, device="cuda"))
    good = np.zeros(T, dtype=bool)
    for e in range(0, 2 * 257, 2):
        good[o[e]:o[e + 1]] = True
    bad = torch.from_numpy(~good).cuda()
    X[bad] = junk
    dY[bad] = junk
    dW = sg.grouped_backward_weight(dY, X, Wg, off).cpu()
    assert sg.grouped_status(Wg) == 0
    Xf[~good] = dYf[~good] = 0.0
    ref = experts.grouped_backward_weight(dYf, Xf, o)[0]
    want = torch.from_numpy(ref).float().to(torch.bfloat16)
    for e in range(0, 2 * 257, 2):
        assert torch.equal(dW[e], want[e]), f"{rows[e]} rows"
