"""The whole expert layer where its kernels can go wrong: numbers near the end of their range, and each way in which the down
kernel deals its steps, with sums that are exact."""
import os
import re

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


MOE = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_gemm_b200", "csrc", "moe.cu")).read()


def down_schedule(fp8, T, E, k, H, I):
    """(groups of eight tokens, CTAs a tile, whether the warps read side by side) of the down kernel, by the rules of moe.cu on
    148 SMs; the expressions that they stand in are looked for, so that a change of them shows here."""
    for rule in ("rows <= kRows ? run<F8, 1>(a, s) : rows <= 2 * kRows ? run<F8, 2>(a, s) : run<F8, 4>(a, s)",
                 "while (parts < 8 && 2 * parts * tiles <= ctas_an_sm * num_sms()) parts *= 2;", "if (steps < 4 * workers) {",
                 "down_ctas(bool f8, int NT) { return light(f8, NT) ? 4 : 2; }", "light(bool f8, int NT) { return !f8 && NT == 1; }",
                 "step_of() { return F8 ? 128 : 64; }"):
        assert rule in re.sub(r"\s+", " ", MOE), rule
    rows = min(T, -(-T * k // E))
    NT = 1 if rows <= 8 else 2 if rows <= 16 else 4
    ctas = 4 if not fp8 and NT == 1 else 2
    parts, tiles = 1, -(-H // 16)
    while parts < 8 and 2 * parts * tiles <= ctas * 148:
        parts *= 2
    return NT, parts, -(-I // (128 if fp8 else 64)) >= 4 * 8 * parts


# several groups a call, steps that the workers do not divide evenly, H and I that end inside a tile and a step
DOWN = [(False, 1, 8, 2, 4104, 4200, (1, 2, True)), (False, 5, 8, 3, 4104, 4664, (1, 2, True)), (False, 8, 6, 2, 4808, 2104, (1, 1, True)),
        (False, 20, 3, 2, 2408, 2104, (2, 1, True)), (False, 20, 3, 2, 1208, 4200, (2, 2, True)), (False, 24, 4, 2, 600, 8264, (2, 4, True)),
        (False, 64, 3, 1, 2408, 2168, (4, 1, True)), (False, 50, 4, 2, 1208, 4232, (4, 2, True)), (False, 3, 5, 2, 4104, 4008, (1, 2, False)),
        (True, 1, 8, 2, 4112, 4112, (1, 1, True)), (True, 8, 6, 3, 2416, 5200, (1, 1, True)), (True, 4, 3, 2, 2064, 8208, (1, 2, True)),
        (True, 20, 3, 2, 2416, 4240, (2, 1, True)), (True, 24, 4, 2, 1200, 8336, (2, 2, True)), (True, 64, 3, 1, 2416, 4112, (4, 1, True)),
        (True, 50, 4, 2, 1216, 8208, (4, 2, True)), (True, 3, 5, 2, 2064, 7952, (1, 2, False)), (True, 40, 2, 1, 80, 528, (4, 8, False))]


@pytest.mark.parametrize("fp8,T,E,k,H,I,schedule", DOWN)
def test_no_step_is_lost_or_doubled(fp8, T, E, k, H, I, schedule):
    """Whole numbers throughout: gates of 128, whose silu is 128 in fp32 (exp(-128) is under 2^-150), features 128 times a sum of
    four whole numbers from -2 to 2, weights of choices that are powers of two, and down weights from -2 to 2; scales by
    tile are powers of two.  Every sum is exact (below 2^24), and every feature counts."""
    assert down_schedule(fp8, T, E, k, H, I) == schedule
    gen = torch.Generator(device="cuda").manual_seed(T * 7 + I)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=gen, device="cuda").to(torch.bfloat16)
    X = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    X.scatter_(1, torch.stack([torch.randperm(H, generator=gen, device="cuda")[:4] for _ in range(T)]), 1.0)
    W13 = torch.cat([torch.full((E, I, H), 32.0, dtype=torch.bfloat16, device="cuda"), draw(-2, 3, E, I, H)], dim=1)
    W2 = draw(-2, 3, E, H, I)
    e = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)]).int()
    e[T // 2, k - 1] = e[T // 2, 0]                      # chosen twice, or the only choice
    w = torch.pow(2.0, torch.randint(-2, 2, (T, k), generator=gen, device="cuda").float())
    w[T // 2] = w[T // 2, 0].clone()
    f13, f2 = W13.double(), W2.double()
    if fp8:
        up_first = I // 128                              # (a tile may hold gate and up rows)
        s13 = torch.ones(E, -(-2 * I // 128), -(-H // 128), device="cuda")
        s13[:, up_first + 1:] = torch.pow(2.0, torch.randint(-1, 2, s13[:, up_first + 1:].shape, generator=gen, device="cuda").float())
        s2 = torch.pow(2.0, torch.randint(-1, 2, (E, -(-H // 128), -(-I // 128)), generator=gen, device="cuda").float())
        spread = lambda s, R, C: s.double().repeat_interleave(128, 1)[:, :R].repeat_interleave(128, 2)[:, :, :C]
        f13, f2 = f13 * spread(s13, 2 * I, H), f2 * spread(s2, H, I)
        a, b = sg.Fp8Tensor(W13.to(torch.float8_e4m3fn), s13), sg.Fp8Tensor(W2.to(torch.float8_e4m3fn), s2)
    else:
        a, b = sg.GroupedWeight(W13), sg.GroupedWeight(W2)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for i in range(E):
            share = w[t][e[t] == i].double().sum()
            if share:
                gate, up = (f13[i] @ X[t].double()).chunk(2)
                assert (gate == 128).all()
                h = share * 128 * up
                assert torch.equal(h, h.to(torch.bfloat16).double())
                want[t] += f2[i] @ h
    got = sg.moe_forward(X, a, b, e, w)
    assert torch.equal(got, want.float().to(torch.bfloat16)) and want.abs().max() < 2 ** 24
    assert got.any(dim=1).all()
    for _ in range(3):
        assert torch.equal(sg.moe_forward(X, a, b, e, w), got)
