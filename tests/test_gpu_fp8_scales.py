"""8-bit products under scales far from one: the product of a row's and a tile's scale is one fp32 number, up to the ends of
its range, on every kernel and in both directions, against the oracle in 64 bits.

Bound: that of tests/_experts.py, and in the subnormal range the rounding of a product of scales, 2^-150 at most, times the sum of
the absolute products of codes, a rounding of 2^-150 for each block's scaled sum and each addition of it, and half a step of
bf16, 2^-134."""
import numpy as np
import pytest
import torch

from oracle import experts
from tests._fp8 import kernel_of
from tests.test_gpu_fp8 import E4M3

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg

KERNELS = [(3, "rows8"), (3, "few"), (40, "few"), (64, "few"), (300, "many")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def tensor(codes, scales):
    return sg.Fp8Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales.astype(np.float32)).cuda())


def calls(T, kernel, A, As, W, Ws):
    """Rows [T, depth] and a weight [cols, depth] of code bytes, with scales by row and by tile, on the wanted kernel: forward
    and input gradient, as far as they take it."""
    outs = []
    if kernel_of(T, 1, W.shape[0]) == kernel:
        outs.append(sg.forward_fp8(tensor(A, As), tensor(W, Ws)))
    if kernel_of(T, 1, W.shape[0], True) == kernel:
        outs.append(sg.backward_input_fp8(tensor(A, As), tensor(np.ascontiguousarray(W.T), np.ascontiguousarray(Ws.T))))
    assert outs
    return [y.double().cpu().numpy() for y in outs]


def product(T, kernel, A, As, W, Ws):
    a, w = E4M3[A], E4M3[W]
    ref, S = experts.fp8_product(a, As.astype(np.float32), w, Ws.astype(np.float32))
    bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * ((A.shape[1] / 16 + 8) * 2.0 ** -22 * S + 2.0 ** -150 * (np.abs(a) @ np.abs(w).T))
    bound += 2.0 ** -134 + 4 * As.shape[1] * 2.0 ** -150
    for got in calls(T, kernel, A, As, W, Ws):
        bad = ~(np.abs(got - ref) <= bound)
        assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[0], got[bad][0], ref[bad][0])
    return ref


def pick(rng, *shape):
    return rng.choice(np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8), shape)


@pytest.mark.parametrize("low,high", [(-77, -60), (-63, -50), (-60, 40), (-20, 50), (-120, 10)])
@pytest.mark.parametrize("T,kernel", KERNELS)
def test_scales_far_apart(T, kernel, low, high):
    """Another scale for each row, tile and block, of either sign, from one size of products to another."""
    rng = np.random.default_rng(T)
    K, N = 400, 272
    draw = lambda *shape: np.ldexp(rng.uniform(1, 2, shape), rng.integers(low, high, shape)) * rng.choice([-1, 1], shape)
    product(T, kernel, pick(rng, T, K), draw(T, 4), pick(rng, N, K), draw(3, 4))


@pytest.mark.parametrize("exponent", [-60, -63, -66, -70, -73, -76])
@pytest.mark.parametrize("T,kernel", KERNELS)
def test_products_of_scales_below_the_normal_numbers(T, kernel, exponent):
    """One size of scales throughout: normal products at 2^-60 each, multiples of 2^-149 further down, and none at 2^-76."""
    rng = np.random.default_rng(T)
    K, N = 144, 272
    A, W = (np.where(rng.random(s) < 0.1, 0x7D, 0x7E).astype(np.uint8) for s in ((T, K), (N, K)))   # 416 and 448
    draw = lambda *shape: np.ldexp(rng.uniform(1, 1.25, shape), exponent)
    As, Ws = draw(T, 2), draw(3, 2)
    product(T, kernel, A, As, W, Ws)
    if exponent == -76:
        assert not any(y.any() for y in calls(T, kernel, A, As, W, Ws))


@pytest.mark.parametrize("T,kernel", KERNELS)
def test_large_scales(T, kernel):
    """Products of scales up to the largest numbers, over sums of zero and over the smallest products of codes."""
    rng = np.random.default_rng(T)
    K, N = 256, 272
    A, W = pick(rng, T, K), pick(rng, N, K)
    A[:, 0:128:2] = 0
    W[:, 1:128:2] = 0                               # the first block's sums are all zero
    As, Ws = rng.uniform(0.5, 1, (T, 2)) * 1e-3, rng.uniform(0.5, 1, (3, 2)) * 1e-3
    As[:, 0], Ws[:, 0] = np.ldexp(1.9, 63), np.ldexp(1.9, np.array([10, 62, 63]))   # up to 3.61 x 2^126
    assert product(T, kernel, A, As, W, Ws).any()
    A[:], W[:] = 0, 0
    A[:, 5], W[:, 5] = 1, 0x81                      # 2^-9 and -2^-9
    assert (product(T, kernel, A, As, W, Ws) < -2.0 ** 54).all()


@pytest.mark.parametrize("T,kernel", KERNELS)
def test_zero_infinite_and_nan_scales(T, kernel):
    """Each stays what it is in a product, and so does a product above the largest number."""
    A, W = np.full((T, 256), 0x38, dtype=np.uint8), np.full((272, 256), 0x38, dtype=np.uint8)   # ones
    As, Ws = np.ones((T, 2)), np.ones((3, 2))
    for a, b, want in ((0.0, 1e30, 128.0), (1e-40, 0.0, 128.0), (np.inf, 1.0, np.inf), (np.inf, 0.0, np.nan), (np.nan, 1e30, np.nan),
                       (1e30, np.nan, np.nan), (1e30, 1e30, np.inf), (-1e30, 1e30, -np.inf)):
        As[:, 1], Ws[:, 1] = a, b
        for y in calls(T, kernel, A, As, W, Ws):
            assert np.array_equal(y, np.full_like(y, want), equal_nan=True), (a, b)
