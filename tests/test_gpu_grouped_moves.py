"""Moves and casts of the expert layer: the handle on the weight follows the parameter."""
import gc

import numpy as np
import pytest
import torch

from tests._experts import normal, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def test_memory_goes_with_the_module():
    gc.collect()
    before = torch.cuda.memory_allocated()
    layer = sg.GroupedLinear(torch.zeros(2, 1024, 1024, dtype=torch.bfloat16, device="cuda"))
    gc.collect()
    assert torch.cuda.memory_allocated() - before >= 4 << 20
    layer.cpu()
    gc.collect()
    assert torch.cuda.memory_allocated() == before


def test_moved_and_back():
    rng = np.random.default_rng(61)
    layer = sg.GroupedLinear(normal(rng, (2, 72, 40))[0], normal(rng, (2, 72))[0])
    X, off = normal(rng, (9, 40))[0], offsets_of([4, 5])[0]
    want = layer(X, off)
    kept = layer.packed
    layer.cuda()
    layer.bfloat16()
    assert layer.packed is kept                     # nothing moved
    layer.cpu()
    with pytest.raises(TypeError):
        layer(X, off)
    layer.cuda()
    assert torch.equal(layer(X, off), want) and sg.grouped_status(layer.packed) == 0
    layer.float()
    with pytest.raises(TypeError):                  # the layer is a bf16 one
        layer(X, off)
    layer.bfloat16()
    assert torch.equal(layer(X, off), want)
