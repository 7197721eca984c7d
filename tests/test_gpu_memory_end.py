"""Inputs and outputs that end with the memory they were cut from: nothing is read or written behind a
tensor's last element, whatever part of a tile lies there."""
import numpy as np
import pytest
import torch

from oracle import experts
from tests._experts import check, integers, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg

SEGMENT = 16 << 20     # an allocation of its own, a whole number of pages


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def at_end(t):
    """A copy of t in the last bytes of an allocation, as near its end as a 16-byte boundary allows."""
    n = t.numel() * t.element_size()
    first = (SEGMENT - n) // 16 * 16
    view = torch.zeros(SEGMENT, dtype=torch.uint8, device="cuda")[first:first + n].view(t.dtype).view(t.shape)
    return view.copy_(t)


CASES = [
    # rows of the experts, N, K, rows before and behind them
    ([67, 1], 72, 1976, 1, 3), ([67, 1], 72, 1976, 0, 0), ([1], 8, 8, 0, 0), ([5], 264, 72, 0, 0), ([33, 0, 2], 136, 200, 0, 0),
    ([129, 0], 520, 1000, 0, 1), ([16, 17, 15], 96, 40, 2, 0), ([255, 130], 24, 648, 0, 0), ([2, 0, 9], 1032, 24, 0, 2),
]


@pytest.mark.parametrize("rows,N,K,first,spare", CASES)
def test_expert_calls(rows, N, K, first, spare):
    rng = np.random.default_rng(81)
    E, T = len(rows), first + sum(rows) + spare
    off, o = offsets_of(rows, first)
    (X, Xf), (W, Wf), (dY, dYf), (b, bf) = (integers(rng, s) for s in ((T, K), (E, N, K), (T, N), (E, N)))
    X, W, dY, b, off = (at_end(t) for t in (X, W, dY, b, off))
    Wg = sg.GroupedWeight(W)
    new = lambda *s: at_end(torch.zeros(*s, dtype=torch.bfloat16, device="cuda"))
    Y = sg.grouped_forward(X, Wg, off, bias=b, out=new(T, N))
    dX = sg.grouped_backward_input(dY, Wg, off, out=new(T, K))
    dW = sg.grouped_backward_weight(dY, X, Wg, off, out=new(E, N, K))
    db = sg.grouped_bias_grad(dY, off, out=new(E, N))
    assert sg.grouped_status(Wg) == 0
    for got, (ref, _) in ((Y, experts.grouped_forward(Xf, Wf, o, bf)), (dX, experts.grouped_backward_input(dYf, Wf, o)),
                          (dW, experts.grouped_backward_weight(dYf, Xf, o)), (db, experts.grouped_bias_grad(dYf, o))):
        assert torch.equal(got.cpu(), torch.from_numpy(ref).float().to(torch.bfloat16))


@pytest.mark.parametrize("rows,N,K", [([67, 1], 72, 1984), ([3], 8, 32), ([33, 0, 2], 136, 224), ([200], 264, 96), ([5, 9], 520, 544)])
def test_4_bit_calls(rows, N, K):
    rng = np.random.default_rng(82)
    E, T = len(rows), sum(rows)
    off, o = offsets_of(rows)
    X, W = at_end(integers(rng, (T, K))[0]), at_end(integers(rng, (E, N, K))[0])
    q = lambda *s: sg.Mx4Tensor(*(at_end(torch.zeros(*s[:-1], s[-1] // d, dtype=torch.uint8, device="cuda")) for d in (2, 32)))
    Xq, Wq = sg.quantize_mx4(X, out=q(T, K)), sg.quantize_mx4(W, out=q(E, N, K))
    back = sg.dequantize_mx4(Xq, out=at_end(X))
    values = lambda t: experts.mx4_values(t.codes.cpu().numpy(), t.scales.cpu().numpy())
    Xf, Wf = values(Xq), values(Wq)
    assert np.array_equal(back.double().cpu().numpy(), Xf)
    new = lambda: at_end(torch.zeros(T, N, dtype=torch.bfloat16, device="cuda"))
    Y = sg.grouped_forward_mx4(Xq, Wq, off, out=new())
    assert torch.equal(Y, sg.grouped_forward_mx4(X, Wq, at_end(off), out=new())) and sg.mx4_status(Wq) == 0
    check(Y, *experts.grouped_forward(Xf, Wf, o), K, "mx4")
