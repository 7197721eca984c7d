"""8-bit and whole-layer calls at the edges of their kernels: weights and rows past 2^31 bytes, sums that CTAs of a cluster
share, chains without waits with weights made just before, and trained routing end to end."""
import numpy as np
import pytest
import torch

from oracle import experts
from tests._experts import check, normal, offsets_of
from tests.test_gpu_fp8 import host, reference, rows_of, weights

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()
    yield
    torch.cuda.empty_cache()


def codes(seed, *shape):
    """Whole numbers -2 .. 2 as e4m3."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in t.flatten(0, -2).split(1 << 14):
        part.copy_(torch.randint(-2, 3, part.shape, generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16))
    return t


def ones(*shape):
    return torch.ones(shape, dtype=torch.float32, device="cuda")


def exact(a, w):
    """bf16 of the exact sums of whole numbers (below 2^24, so that fp32 holds them)."""
    return (a.float().double() @ w.float().double()).float().to(torch.bfloat16)


def test_far_rows_and_far_outputs():
    """Rows, outputs and scales past 2^31 elements, on the tiles of many rows."""
    K, N, T = 8192, 16, 270000
    X = codes(1, T, K)
    q = sg.Fp8Tensor(X, ones(T, K // 128))
    W = codes(2, N, K)
    Wq = sg.Fp8Tensor(W, ones(1, K // 128))
    Y = sg.forward_fp8(q, Wq)
    for a in range(0, T, 54000):
        assert torch.equal(Y[a:a + 54000], exact(X[a:a + 54000], W.float().T)), a
    dY = codes(3, T, N)
    dX = sg.backward_input_fp8(sg.Fp8Tensor(dY, ones(T, 1)), Wq)
    assert dX.numel() > 2 ** 31
    for a in (0, 131000, T - 300):
        assert torch.equal(dX[a:a + 300], exact(dY[a:a + 300], W.float())), a
    back = sg.quantize_fp8(sg.dequantize_fp8(q))          # bf16 and back, at scale 2 / 448 or 1 / 448 ...
    for a in (0, T - 1000):
        assert torch.equal(sg.dequantize_fp8(sg.Fp8Tensor(back.codes[a:a + 1000].contiguous(), back.scales[a:a + 1000].contiguous())).float(),
                           X[a:a + 1000].float())


@pytest.mark.parametrize("T", [6, 40, 700])
def test_far_experts(T):
    """Weights of more than 2^31 elements: the last experts' planes, each kernel, both directions, and the whole layer."""
    E, N, K = 40, 8192, 8192
    W = codes(4, E, N, K)
    Wq = sg.Fp8Tensor(W, ones(E, N // 128, K // 128))
    rows = [0] * E
    rows[0], rows[E - 1] = T // 2, T - T // 2
    off, o = offsets_of(rows)
    X, dY = codes(5, T, K), codes(6, T, N)
    Y = sg.grouped_forward_fp8(sg.Fp8Tensor(X, ones(T, K // 128)), Wq, off)
    dX = sg.grouped_backward_input_fp8(sg.Fp8Tensor(dY, ones(T, N // 128)), Wq, off)
    for e in (0, E - 1):
        r = slice(int(o[e]), int(o[e + 1]))
        assert torch.equal(Y[r], exact(X[r], W[e].float().T)), e
        assert torch.equal(dX[r], exact(dY[r], W[e].float())), e
    assert sg.fp8_status(Wq) == 0
    if T > 6:
        return
    # a whole layer of the same weights: [E, 2 I, H] of 8192 x 8192, and 8192 x 4096 of them as the down weights
    W2 = W.view(E, 2 * N, K // 2)[:, :N].contiguous()
    W2q = sg.Fp8Tensor(W2, ones(E, N // 128, K // 2 // 128))
    x = (0.01 * torch.randn(T, K, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")).to(torch.bfloat16)
    e = torch.tensor([[0, E - 1]] * T, dtype=torch.int32, device="cuda")
    w = torch.full((T, 2), 0.5, device="cuda")
    got = sg.moe_forward(x, Wq, W2q, e, w).double()
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for i in (0, E - 1):
        z = x.double() @ W[i].float().double().T
        h = torch.nn.functional.silu(z[:, :N // 2]) * z[:, N // 2:]
        want += 0.5 * (h @ W2[i].float().double().T)
    # h is rounded by 2^-8, each of 2 x 4096 terms with its own sign: 2^-8 of the root of their squares, six times, and y
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 6 * 2.0 ** -8 * want.std() + 1e-3 * want.abs().max()).all()


@pytest.mark.parametrize("M,K,N", [(9, 4112, 24), (16, 1024, 128), (17, 2064, 136), (33, 3968, 8), (48, 528, 264), (64, 8208, 120),
                                   (200, 2064, 512), (255, 4096, 1024)])
def test_clusters_that_cut_the_blocks(M, K, N):
    """Few tiles: two to eight CTAs share one, the blocks do not divide evenly."""
    rng = np.random.default_rng(M)
    X, q, xr = rows_of(rng, M, K)
    Wq, wr = weights(rng, N, K)
    bias, bf = normal(rng, (N,))
    Y = sg.forward_fp8(X, Wq, bias=bias)
    check(Y, *reference(xr, wr, bias=bf), K, "forward")
    assert all(torch.equal(Y, sg.forward_fp8(q, Wq, bias=bias)) for _ in range(3))
    W2, w2 = weights(rng, K // 16 * 16, max(16, N // 16 * 16))
    g, gq, gr = rows_of(rng, M, K // 16 * 16)
    check(sg.backward_input_fp8(g, W2), *reference(gr, w2, transposed=True), K, "gradient")


@pytest.mark.parametrize("rows", [[3, 0, 4], [12, 0, 30], [64, 65, 0], [90, 200, 150]])
def test_chain_without_waits(rows):
    """Weights quantised and multiplied at once, rows that the call before wrote, offsets made by the router: eager, and as
    a replayed graph, against the same calls with a wait behind each."""
    E, D, steps = 3, 256, 4
    rng = np.random.default_rng(sum(rows))
    T = sum(rows)
    logits = torch.full((T, E), -9.0, device="cuda")
    owner = rng.permutation(np.repeat(np.arange(E), rows))
    logits[torch.arange(T), torch.from_numpy(owner).cuda()] = 1.0
    banks = [normal(rng, (E, D, D), D ** -0.5)[0] for _ in range(steps)]
    X0 = normal(rng, (T, D))[0]
    Wq = sg.quantize_fp8(banks[0], block_rows=128)
    Wq.status
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    A, B, X = torch.empty_like(X0), torch.empty_like(X0), X0.clone()
    G = [torch.empty_like(X0) for _ in range(steps)]

    def run(wait=lambda: None):
        A.copy_(X)
        for i in range(steps):
            sg.quantize_fp8(banks[i], block_rows=128, out=Wq)
            wait()
            off.copy_(sg.route(logits, 1).offsets)
            wait()
            sg.grouped_forward_fp8(A, Wq, off, out=B)
            wait()
            sg.grouped_backward_input_fp8(B, Wq, off, out=G[i])
            wait()
            sg.grouped_forward_fp8(B, Wq, off, out=A)
            wait()

    results = lambda: [A, B, *G]
    run(torch.cuda.synchronize)
    want = [t.clone() for t in results()]
    assert all(torch.isfinite(t.float()).all() and t.any() for t in want)

    def poison():
        for t in results():
            t.fill_(float("nan"))
        off.fill_(-1)
        torch.cuda.synchronize()

    for rep in range(4):
        poison()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), want)), rep
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(4):
        poison()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), want)), rep
    assert sg.fp8_status(Wq) == 0


def test_routed_layer_trains():
    """Router, sorted rows, bf16 experts and their sum, as the router's documentation has it: forward against the whole
    layer's kernel, gradients of logits, inputs and weights against torch in 64 bits."""
    rng = np.random.default_rng(5)
    T, E, k, D = 50, 6, 2, 64
    X, Xf = normal(rng, (T, D))
    layer = sg.GroupedLinear(normal(rng, (E, D, D), D ** -0.5)[0])
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    X.requires_grad_(True)
    logits.requires_grad_(True)
    r = sg.route(logits, k)
    rows = X[r.order // k]
    y = layer(rows, r.offsets)
    out = torch.zeros_like(X).index_add(0, r.order // k, y * r.weights.flatten()[r.order, None].to(y.dtype))
    g, gf = normal(rng, (T, D))
    out.backward(g)
    # the same in 64 bits
    x64 = torch.from_numpy(Xf).requires_grad_(True)
    l64 = logits.detach().double().cpu().requires_grad_(True)
    w64 = layer.weight.detach().double().cpu().requires_grad_(True)
    e = r.experts.long().cpu()
    p = torch.softmax(l64, 1).gather(1, e)
    w = p / p.sum(1, keepdim=True)
    o64 = torch.einsum("tk,tkn->tn", w, torch.einsum("tknd,td->tkn", w64[e], x64))
    o64.backward(torch.from_numpy(gf))
    # roundings to bf16 of products, weights, sums and gradients: some of 2^-8 of values of this size
    for got, want in ((out, o64), (X.grad, x64.grad), (logits.grad, l64.grad), (layer.weight.grad, w64.grad)):
        want = want.detach()
        diff = (got.detach().double().cpu() - want).abs()
        assert diff.max() <= 8 * 2.0 ** -8 * want.abs().max(), (diff.max(), want.abs().max())


def test_calls_on_two_streams_at_once():
    """The same weights on two streams at once: workspaces and sums are each call's own."""
    rng = np.random.default_rng(6)
    E, T, H, I = 8, 24, 512, 528
    W13 = sg.quantize_fp8(normal(rng, (E, 2 * I, H), H ** -0.5)[0], block_rows=128)
    W2 = sg.quantize_fp8(normal(rng, (E, H, I), I ** -0.5)[0], block_rows=128)
    Xs = [normal(rng, (T, H))[0] for _ in range(2)]
    ls = [torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda() for _ in range(2)]
    W13.status, W2.status

    def layer(i):
        r = sg.route(ls[i], 2)
        y = sg.moe_forward(Xs[i], W13, W2, r.experts, r.weights)
        rows = Xs[i][r.order // 2]
        return y, sg.grouped_forward_fp8(rows, W13, r.offsets), r.order

    want = [layer(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(10):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(layer(i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), rep


@pytest.mark.parametrize("T", [100, 5000])
def test_routers_of_two_graphs_and_their_gradients(T):
    """One CTA, and two kernels with counts between them; the same pool, replayed in turn with other logits."""
    rng = np.random.default_rng(T)
    make = lambda: torch.from_numpy(rng.standard_normal((T, 72)).astype(np.float32)).cuda()
    graphs = []
    for k in (3, 8):
        l, d = make(), torch.ones(T, k, device="cuda")
        sg.route_backward(d, l, sg.route(l, k).experts)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0][0].pool() if graphs else None):
            r = sg.route(l, k, renormalize=False)
            dl = sg.route_backward(r.weights, l, r.experts, renormalize=False)
        graphs.append((g, k, l, r, dl))
    for _ in range(3):
        for g, k, l, r, dl in graphs:
            l.copy_(make())
            g.replay()
            want = sg.route(l, k, renormalize=False)
            assert all(torch.equal(a, b) for a, b in zip(r, want))
            assert torch.equal(dl, sg.route_backward(want.weights, l, want.experts, renormalize=False))


def test_broadcast_and_unused_gradients_of_the_router():
    """The gradient of a sum is a broadcast scalar; weights that nothing uses have a gradient of zeros."""
    l = torch.randn(50, 24, device="cuda").requires_grad_(True)
    r = sg.route(l, 4, score="sigmoid", renormalize=False)
    r.weights.sum().backward()
    assert torch.equal(l.grad, sg.route_backward(torch.ones(50, 4, device="cuda"), l.detach(), r.experts, "sigmoid", False))
    chosen = torch.zeros(50, 24, dtype=torch.bool, device="cuda").scatter_(1, r.experts.long(), True)
    assert not l.grad[~chosen].any() and (l.grad[chosen] > 0).all()
    l.grad = None
    (sg.route(l, 4).weights * 0 + l[:, :4]).sum().backward()
    assert torch.equal(l.grad, torch.ones_like(l) * (torch.arange(24, device="cuda") < 4))


def test_state_dict_assigned_and_moved_buffers():
    """Buffers whose storage is replaced: the handle is made anew, with its status word."""
    rng = np.random.default_rng(21)
    W, _ = normal(rng, (144, 272))
    x, _ = normal(rng, (9, 272))
    a = sg.Fp8Linear.from_dense(W)
    b = sg.Fp8Linear.from_dense(torch.zeros_like(W))
    before = b.weight8
    b.load_state_dict({n: t.clone() for n, t in a.state_dict().items()}, assign=True)
    assert torch.equal(a(x), b(x)) and b.weight8 is not before and sg.fp8_status(b.weight8) == 0
    assert torch.equal(b.to("cpu").to("cuda")(x), a(x))


def test_results_repeat_to_the_bit():
    """Every output is a sum in a fixed order, whatever else the GPU does: clusters, teams and shared sums included."""
    rng = np.random.default_rng(22)
    Wq, _ = weights(rng, 6, 272, 528)
    off, _ = offsets_of([3, 0, 65, 1, 130, 20], 0)
    X, _ = normal(rng, (219, 528))
    W13, W2 = sg.quantize_fp8(normal(rng, (6, 288, 528), 0.05)[0], 128), sg.quantize_fp8(normal(rng, (6, 528, 144), 0.08)[0], 128)
    r = sg.route(torch.randn(40, 6, device="cuda"), 3)
    calls = (lambda: sg.grouped_forward_fp8(X, Wq, off), lambda: sg.forward_fp8(X[:5].contiguous(), sg.Fp8Tensor(Wq.codes[0], Wq.scales[0])),
             lambda: sg.moe_forward(X[:40].contiguous(), W13, W2, r.experts, r.weights))
    first = [c() for c in calls]
    for _ in range(20):
        for c, y in zip(calls, first):
            assert torch.equal(c(), y)
