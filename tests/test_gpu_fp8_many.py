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


SHARES = [([700, 0, 333], 1008, 720), ([1, 0, 800, 257], 272, 400), ([256, 257, 255, 1, 31, 32, 33, 0, 700], 1008, 720),
          ([0, 0, 1100], 528, 272), ([0, 300, 211, 0, 190, 64, 402, 33, 0, 17, 351], 1008, 720), ([90, 513, 290], 128, 1040)]


@pytest.mark.parametrize("rows,K,N", SHARES)
def test_experts(rows, K, N):
    """Both directions, each expert's own weights, scales and bias, tiles that end beside another expert's rows, rows of no
    expert at both ends (NaN there, and left alone in `out`)."""
    rng = np.random.default_rng(sum(rows) + K)
    front, back = 3, 37
    T, E = front + sum(rows) + back, len(rows)
    off, o = offsets_of(rows, front)
    Wq, wr = weights(rng, E, N, K)
    bias, bf = normal(rng, (E, N))
    rest = np.r_[0:front, T - back:T]
    for depth, cols, transposed in ((K, N, False), (N, K, True)):
        assert kernel_of(T, E, cols, transposed) == "many"
        A, _ = normal(rng, (T, depth))
        A[rest] = float("nan")
        q = sg.quantize_fp8(A)
        c, s = host(q)
        c[rest], s[rest] = 0, 0
        call = (lambda a, **kw: sg.grouped_backward_input_fp8(a, Wq, off, **kw)) if transposed else \
            (lambda a, **kw: sg.grouped_forward_fp8(a, Wq, off, bias=bias, **kw))
        Y = call(A)
        check(Y, *reference((c, s), wr, o, transposed, None if transposed else bf), depth, f"transposed {transposed}")
        assert not Y[rest].any()
        assert torch.equal(Y, call(q))
        out = torch.full((T, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        call(A, out=out)
        assert (out[rest] == 7).all() and torch.equal(out[front:T - back], Y[front:T - back])
    assert sg.fp8_status(Wq) == 0


@pytest.mark.parametrize("offsets", [[0, 900, 300, 2000], [-5, 700, 1500, 1100], [1100, 0, 400, 5], [-(2 ** 31), 2 ** 31 - 1, 0, 1100]])
def test_bad_offsets_are_clamped_and_reported(offsets):
    rng = np.random.default_rng(1)
    T = 1100
    Wq, wr = weights(rng, 3, 400, 272)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    safe = np.maximum.accumulate(np.clip(offsets, 0, T))
    for depth, cols, transposed in ((272, 400, False), (400, 272, True)):
        assert kernel_of(T, 3, cols, transposed) == "many"
        A, _ = normal(rng, (T, depth))
        call = sg.grouped_backward_input_fp8 if transposed else sg.grouped_forward_fp8
        check(call(A, Wq, off), *reference(host(sg.quantize_fp8(A)), wr, safe, transposed), depth, "clamped")
        assert sg.fp8_status(Wq) == 1 and sg.fp8_status(Wq) == 0


def test_no_expert_has_rows():
    rng = np.random.default_rng(2)
    Wq, _ = weights(rng, 3, 400, 272)
    for first in (0, 500, 1100):
        off = torch.full((4,), first, dtype=torch.int32, device="cuda")
        for depth, call in ((272, sg.grouped_forward_fp8), (400, sg.grouped_backward_input_fp8)):
            A = torch.full((1100, depth), float("nan"), dtype=torch.bfloat16, device="cuda")
            assert not call(A, Wq, off).any()
    assert sg.fp8_status(Wq) == 0


def test_far_experts_with_their_own_scales():
    """Weights of more than 2^31 elements, uneven shares, the last expert's plane among them; whole numbers and powers of two."""
    E, N, K, T = 40, 8192, 8192, 2700
    rows = [0] * E
    rows[0], rows[17], rows[38], rows[E - 1] = 900, 1, 1300, 499
    assert kernel_of(T, E, N) == kernel_of(T, E, K, True) == "many"
    gen = torch.Generator(device="cuda").manual_seed(4)

    def codes(*shape):
        t = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        for part in t.flatten(0, -2).split(1 << 14):
            part.copy_(torch.randint(-2, 3, part.shape, generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16))
        return t

    power = lambda *shape: torch.pow(2.0, torch.randint(-1, 2, shape, generator=gen, device="cuda").float())
    W, ws = codes(E, N, K), power(E, N // 128, K // 128)
    Wq = sg.Fp8Tensor(W, ws)
    off, o = offsets_of(rows)
    X, xs, dY, gs = codes(T, K), power(T, K // 128), codes(T, N), power(T, N // 128)
    Y = sg.grouped_forward_fp8(sg.Fp8Tensor(X, xs), Wq, off)
    dX = sg.grouped_backward_input_fp8(sg.Fp8Tensor(dY, gs), Wq, off)
    for e in (0, 17, 38, E - 1):
        r = slice(int(o[e]), int(o[e + 1]))
        w = W[e].float().double() * ws[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        x = X[r].float().double() * xs[r].double().repeat_interleave(128, 1)
        g = dY[r].float().double() * gs[r].double().repeat_interleave(128, 1)
        assert torch.equal(Y[r], (x @ w.T).float().to(torch.bfloat16)), e
        assert torch.equal(dX[r], (g @ w).float().to(torch.bfloat16)), e
    assert sg.fp8_status(Wq) == 0


@pytest.mark.parametrize("E,T,most", [(64, 4096, 0.9), (64, 4097, 0.9), (256, 9000, 0.97), (1024, 5000, 0.5), (1024, 66000, 0.99)])
def test_skewed_shares_of_many_experts(E, T, most):
    """One expert with nearly all rows, the others with few or none, on both sides of the rule between the kernels."""
    rng = np.random.default_rng(E + T)
    N, K = 144, 272
    big = int(rng.integers(E))
    rows = rng.multinomial(T - int(most * T), np.full(E, 1 / E))
    rows[big] += int(most * T)
    off, o = offsets_of(rows)
    Wq, wr = weights(rng, E, N, K)
    pick = np.unique(np.r_[0:40, T - 40:T, rng.integers(0, T, 200), o[big] - 3:o[big] + 3, o[big + 1] - 3:o[big + 1] + 3].clip(0, T - 1))
    owner = np.searchsorted(o, pick, side="right") - 1
    for depth, call, transposed in ((K, sg.grouped_forward_fp8, False), (N, sg.grouped_backward_input_fp8, True)):
        A, _ = normal(rng, (T, depth))
        Y = call(A, Wq, off)
        c, s = host(sg.quantize_fp8(A))
        at = np.r_[0, np.cumsum(np.bincount(owner, minlength=E))]
        check(Y[torch.from_numpy(pick).cuda()], *reference((c[pick], s[pick]), wr, at, transposed), depth, f"transposed {transposed}")
        assert torch.isfinite(Y.float()).all()
    assert sg.fp8_status(Wq) == 0


def test_chain_of_experts_without_waits():
    """Weights quantised and multiplied at once on these tiles, rows that the call before wrote: eager and as a replayed graph,
    against the same calls with a wait behind each."""
    E, D, steps = 3, 256, 3
    rng = np.random.default_rng(3)
    rows = [700, 100, 400]
    T = sum(rows)
    assert kernel_of(T, E, D) == "many"
    off, _ = offsets_of(rows)
    banks = [normal(rng, (E, D, D), D ** -0.5)[0] for _ in range(steps)]
    X = normal(rng, (T, D))[0]
    Wq = sg.quantize_fp8(banks[0], block_rows=128)
    Wq.status
    outs = [torch.empty_like(X) for _ in range(2 * steps)]

    def run(wait=lambda: None):
        A = X
        for i in range(steps):
            sg.quantize_fp8(banks[i], block_rows=128, out=Wq)
            wait()
            sg.grouped_forward_fp8(A, Wq, off, out=outs[2 * i])
            wait()
            sg.grouped_backward_input_fp8(outs[2 * i], Wq, off, out=outs[2 * i + 1])
            wait()
            A = outs[2 * i + 1]

    run(torch.cuda.synchronize)
    want = [t.clone() for t in outs]
    assert all(torch.isfinite(t.float()).all() and t.any() for t in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(6):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay() if rep % 2 else run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep
