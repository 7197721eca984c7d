"""Expert and 4-bit calls whose rows, outputs, weight planes or 4-bit rows pass 2^31 elements, sums over
hundreds of thousands of rows, and the edges of the 4-bit tiles.

Inputs of the bf16 products are small integers, so every sum is exact in fp32 and one rounding to
bf16 remains: results are equal to the rounded exact ones, over all rows.
"""
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
    yield
    torch.cuda.empty_cache()


def ints(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in t.flatten(0, -2).split(1 << 15):
        part.copy_(torch.randint(-2, 3, part.shape, generator=gen, device="cuda", dtype=torch.int8))
    return t


def rounded(x):
    """fp64, exact integers below 2^24, to bf16 in one rounding (fp32 holds them)."""
    assert x.abs().max() < 2 ** 24
    return x.float().to(torch.bfloat16)


def same_rows(Y, X, W, first, last, chunk=1 << 14):
    for a in range(first, last, chunk):
        b = min(last, a + chunk)
        assert torch.equal(Y[a:b], rounded(X[a:b].double() @ W.double().T)), (a, b)


def test_long_sums_over_far_rows():
    K, N, T = 8192, 16, 270000
    assert T * K > 2 ** 31
    X, dY = ints(1, T, K), ints(2, T, N)
    Wg = sg.GroupedWeight(ints(3, 2, N, K))
    off = torch.tensor([0, T - 37, T], dtype=torch.int32, device="cuda")
    dW = sg.grouped_backward_weight(dY, X, Wg, off)
    db = sg.grouped_bias_grad(dY, off)
    Y = sg.grouped_forward(X, Wg, off)
    dX = sg.grouped_backward_input(dY, Wg, off)
    assert sg.grouped_status(Wg) == 0
    for e, (a, b) in enumerate(((0, T - 37), (T - 37, T))):
        ref = torch.zeros(N, K, dtype=torch.float64, device="cuda")
        for i in range(a, b, 1 << 14):
            j = min(b, i + (1 << 14))
            ref += dY[i:j].double().T @ X[i:j].double()
        assert torch.equal(dW[e], rounded(ref)), e
        assert torch.equal(db[e], rounded(dY[a:b].double().sum(0))), e
        same_rows(Y, X, Wg.weight[e], a, b)
        same_rows(dX, dY, Wg.weight[e].T, a, b)


@pytest.mark.parametrize("call", ["forward", "input gradient"])
def test_far_outputs(call):
    """Output rows past 2^31 elements, the zeros behind them, and an output whose rows of none stay."""
    T, wide, deep = 270000, 8192, 16
    N, K = (wide, deep) if call == "forward" else (deep, wide)
    A = ints(4, T, deep)
    Wg = sg.GroupedWeight(ints(5, 2, N, K))
    fn = sg.grouped_forward if call == "forward" else sg.grouped_backward_input
    cut, end = 262150, 269000                       # 262144 rows are 2^31 elements
    off = torch.tensor([5, cut, end], dtype=torch.int32, device="cuda")
    Y = fn(A, Wg, off)
    assert sg.grouped_status(Wg) == 0
    for e, (a, b) in enumerate(((5, cut), (cut, end))):
        same_rows(Y, A, Wg.weight[e] if call == "forward" else Wg.weight[e].T, a, b)
    assert not Y[:5].any() and not Y[end:].any()
    out = torch.full_like(Y, 7.0)
    fn(A, Wg, off, out=out)
    assert torch.equal(out[5:end], Y[5:end]) and (out[:5] == 7.0).all() and (out[end:] == 7.0).all()


@pytest.mark.parametrize("rows", [3, 12, 300])
def test_far_weight_planes(rows):
    E, N, K = 9, 16384, 16384
    assert (E - 1) * N * K >= 2 ** 31
    Wg = sg.GroupedWeight(ints(6, E, N, K))
    per = [rows] + [0] * (E - 2) + [rows]
    off, T = offsets_of(per)[0], 2 * rows
    X, dY, bias = ints(7, T, K), ints(8, T, N), ints(9, E, N)
    Y = sg.grouped_forward(X, Wg, off, bias=bias)
    dX = sg.grouped_backward_input(dY, Wg, off)
    for e, r in ((0, slice(0, rows)), (E - 1, slice(rows, T))):
        W = Wg.weight[e].double()
        assert torch.equal(Y[r], rounded(X[r].double() @ W.T + bias[e].double()))
        assert torch.equal(dX[r], rounded(dY[r].double() @ W))
        del W
    dW = sg.grouped_backward_weight(dY, X, Wg, off)
    db = sg.grouped_bias_grad(dY, off)
    assert sg.grouped_status(Wg) == 0
    for e, r in ((0, slice(0, rows)), (E - 1, slice(rows, T))):
        assert torch.equal(dW[e], rounded(dY[r].double().T @ X[r].double()))
        assert torch.equal(db[e], rounded(dY[r].double().sum(0)))
    for e in range(1, E - 1):
        assert not dW[e].any() and not db[e].any()


def values(q, rows):
    return experts.mx4_values(q.codes[rows].cpu().numpy(), q.scales[rows].cpu().numpy())


def test_far_4_bit_rows():
    T, K, N = 66000, 32768, 264
    assert T * K > 2 ** 31
    rng = np.random.default_rng(71)
    X = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    X.normal_(generator=torch.Generator(device="cuda").manual_seed(10))
    q = sg.quantize_mx4(X)
    back = sg.dequantize_mx4(q)
    for a in range(0, T, 1 << 13):                  # no row's bits depend on where it lies
        part = sg.quantize_mx4(X[a:a + (1 << 13)])
        assert torch.equal(q.codes[a:a + (1 << 13)], part.codes) and torch.equal(q.scales[a:a + (1 << 13)], part.scales)
        assert torch.equal(back[a:a + (1 << 13)], sg.dequantize_mx4(part))
    Wq = sg.quantize_mx4(normal(rng, (N, K), K ** -0.5)[0])
    Y = sg.forward_mx4(X, Wq)
    assert torch.equal(Y, sg.forward_mx4(q, Wq)) and sg.mx4_status(Wq) == 0
    rows = [0, 1, 65530, 65535, 65536, 65537, T - 100, T - 1]     # 65536 rows are 2^31 elements
    Xf, Wf = values(q, rows), values(Wq, slice(None))
    check(Y[rows], Xf @ Wf.T, np.abs(Xf) @ np.abs(Wf).T, K, "rows")


@pytest.mark.parametrize("rows", [2, 40])
def test_far_4_bit_weight_planes(rows):
    E, N, K = 9, 16384, 16384
    W = ints(11, E, N, K)
    Wq = sg.quantize_mx4(W)
    del W
    off = offsets_of([rows] + [0] * (E - 2) + [rows])[0]
    X = normal(np.random.default_rng(72), (2 * rows, K))[0]
    Y = sg.grouped_forward_mx4(X, Wq, off)
    assert sg.mx4_status(Wq) == 0
    Xf = values(sg.quantize_mx4(X), slice(None))
    cols = slice(N - 300, N)
    for e, r in ((0, slice(0, rows)), (E - 1, slice(rows, 2 * rows))):
        Wf = values(Wq, (e, cols))
        check(Y[r, cols], Xf[r] @ Wf.T, np.abs(Xf[r]) @ np.abs(Wf).T, K, f"expert {e}")


def tile_edges(rows, most, step=32):
    """First and last row of each tile when rows are cut into the fewest tiles of at most `most`, spread
    evenly in units of `step`."""
    tiles, units = -(-rows // most), -(-rows // step)
    q, more = divmod(units, tiles)
    first = [(i * q + min(i, more)) * step for i in range(tiles)]
    return sorted({r for f in first for r in (f - 1, f) if r >= 0} | {rows - 1})


@pytest.mark.parametrize("M,N,K", [(3000, 520, 1024), (1500, 1032, 1312), (9000, 264, 544), (193, 264, 96), (385, 136, 512),
                                   (577, 264, 2080)])
def test_edges_of_the_4_bit_tiles(M, N, K):
    rng = np.random.default_rng(M)
    Wq = sg.quantize_mx4(normal(rng, (N, K), K ** -0.5)[0])
    Xq = sg.quantize_mx4(normal(rng, (M, K))[0])
    Y = sg.forward_mx4(Xq, Wq)
    rows = tile_edges(M, 192)
    assert len(rows) >= 2 * (M // 192)
    Xf, Wf = values(Xq, rows), values(Wq, slice(None))
    check(Y[rows], Xf @ Wf.T, np.abs(Xf) @ np.abs(Wf).T, K, "edges")
    assert sg.mx4_status(Wq) == 0
