"""The whole expert layer where its kernels can go wrong: numbers near the end of their range."""
import numpy as np
import pytest
import torch

from oracle import experts as oracle
from tests._experts import normal
from tests.test_gpu_route_moe import Layer, assert_layer, choices

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def scaled(rng, E, H, I, fp8, std13, std2):
    """A layer with weights of these sizes."""
    layer = Layer(rng, E, 16, 16, fp8)
    w13, f13 = normal(rng, (E, 2 * I, H), std13)
    w2, f2 = normal(rng, (E, H, I), std2)
    layer.H, layer.I = H, I
    if fp8:
        layer.W13, layer.W2 = (sg.quantize_fp8(w, block_rows=128) for w in (w13, w2))
        layer.values()
    else:
        layer.W13, layer.W2, layer.f13, layer.f2 = sg.GroupedWeight(w13), sg.GroupedWeight(w2), f13, f2
    return layer


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 9, 40])
@pytest.mark.parametrize("std,std13,std2", [(1e18, 0.06, 0.08), (1e36, 3e-30, 0.08), (1e36, 1e-19, 1e-6), (1e-15, 0.06, 0.08)])
def test_large_and_small_numbers(T, std, std13, std2, fp8):
    """Inputs and features up to 10^36, whose sums of products with codes (up to 448) would leave fp32 though those with the
    weights do not; and small ones."""
    rng = np.random.default_rng(T)
    layer = scaled(rng, 3, 272, 144, fp8, std13, std2)
    X, Xf = normal(rng, (T, 272), std)
    e, w, ef, wf = choices(rng, T, 3, 2)
    Y = sg.moe_forward(X, layer.W13, layer.W2, e, w)
    ref, _ = oracle.moe_forward(Xf, layer.f13, layer.f2, ef, wf)
    assert np.abs(ref).max() < 3e38 and ref.any()
    assert_layer(Y, Xf, layer, ef, wf)
