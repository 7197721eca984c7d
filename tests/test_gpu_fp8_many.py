"""The 8-bit products on the tiles of many rows, by expert: planes of weights, scales and bias, tiles that end beside another
expert's rows, rows of no expert, clamped offsets, far planes, and the scales' ring in shared memory."""
import numpy as np
import pytest
import torch

from tests._experts import check, normal, offsets_of
from tests._fp8 import kernel_of
from tests.test_gpu_fp8 import host, reference, weights

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("depth,N", [(16, 272), (128, 1032), (256, 4360), (384, 2064), (896, 1024), (4112, 1032)])
@pytest.mark.parametrize("transposed", [False, True])
def test_every_block_meets_its_own_scales(depth, N, transposed):
    """Codes of one, whole numbers as scales, another for each row and block: sums are exact (below 2^24), and a stage that
    read another stage's scales would show.  Several tiles a CTA, one block a tile and many; again and again."""
    T, cols = 2300, N // 16 * 16 if transposed else N
    assert kernel_of(T, 1, cols, transposed) == "many"
    nb, nc = -(-depth // 128), -(-cols // 128)
    t, b, c = (torch.arange(n, device="cuda") for n in (T, nb, nc))
    rs = (1 + (7 * t[:, None] + 3 * b) % 5).float()
    ws = (1 + (c[:, None] + b) % 3).float()
    one = lambda *shape: torch.ones(shape, dtype=torch.bfloat16, device="cuda").to(torch.float8_e4m3fn)
    q = sg.Fp8Tensor(one(T, depth), rs)
    if transposed:
        Wq, call = sg.Fp8Tensor(one(depth, cols), ws.T.contiguous()), sg.backward_input_fp8
    else:
        Wq, call = sg.Fp8Tensor(one(cols, depth), ws), sg.forward_fp8
    width = (depth - 128 * b).clamp(max=128).double()
    want = ((rs.double() * width) @ ws.double().T).repeat_interleave(128, dim=1)[:, :cols].to(torch.bfloat16)
    for rep in range(10):
        assert torch.equal(call(q, Wq), want), rep
    assert sg.fp8_status(Wq) == 0
