"""GPU parity of the router and of the whole expert layer for a few tokens against the fp64 oracle, and of the two
together with the grouped products."""
import numpy as np
import pytest
import torch

from oracle import experts as oracle
from tests._experts import normal
from tests.test_gpu_fp8 import E4M3, host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


# ---------------------------------------------------------------- router


def logits_of(rng, T, E, half=False, std=2.0):
    """(CUDA logits, fp64): bf16 ones have many equal neighbours."""
    t = torch.from_numpy((rng.standard_normal((T, E)) * std).astype(np.float32)).cuda()
    t = t.to(torch.bfloat16) if half else t
    return t, t.double().cpu().numpy()


def eps_of(E, f):
    """Relative error of a weight: two exponentials (2^-22 each, and 2^-24 of the argument, a rounded difference), sums
    of up to E / 32 + 5 additions, a division and a product."""
    finite = f[np.isfinite(f)]
    spread = float(finite.max() - finite.min()) if finite.size else 0.0
    return 2 * (2.0 ** -22 + spread * 2.0 ** -24) + (E / 32 + 5 + 4) * 2.0 ** -24


def assert_routed(r, f, k, sort=True, **how):
    e, w, offsets, order = oracle.route(f, k, **how)
    assert np.array_equal(r.experts.cpu().numpy(), e)
    got = r.weights.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(w))
    some = ~np.isnan(w)
    # (below 2^-126 a score is rounded to steps of 2^-149 or to zero)
    assert (np.abs(got - w)[some] <= eps_of(f.shape[1], f) * np.abs(w)[some] + 2.0 ** -126 * abs(how.get("factor", 1.0))).all()
    if sort:
        assert np.array_equal(r.offsets.cpu().numpy(), offsets)
        assert np.array_equal(r.order.cpu().numpy(), order)
    else:
        assert r.offsets is None and r.order is None


HOW = [dict(score="softmax", renormalize=True), dict(score="softmax", renormalize=False, factor=2.5),
       dict(score="sigmoid", renormalize=True, factor=0.7), dict(score="sigmoid", renormalize=False)]


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 8, 8), (8, 33, 3), (61, 64, 6), (128, 40, 5), (129, 16, 4), (200, 300, 8),
                                   (1000, 128, 8), (37, 1024, 32), (131, 1000, 32)])
def test_route(T, E, k, how):
    rng = np.random.default_rng(T + E)
    for half in (False, True):
        l, f = logits_of(rng, T, E, half)
        assert_routed(sg.route(l, k, **how), f, k, **how)
        assert_routed(sg.route(l, k, sort=False, **how), f, k, sort=False, **how)


def test_route_of_a_long_prompt():
    """Runs of several tokens a warp, many CTAs; an expert with nearly all tokens, experts without any."""
    rng = np.random.default_rng(1)
    l, f = logits_of(rng, 20011, 96)
    l[:, 17] += 6
    l[:, 40:50] = -float("inf")
    f = l.double().cpu().numpy()
    assert_routed(sg.route(l, 4), f, 4)


@pytest.mark.parametrize("T,E,k", [(131073, 8, 2), (300001, 12, 3), (140000, 40, 32)])
def test_route_of_very_many_tokens(T, E, k):
    """Runs longer than 128 tokens, up to what a CTA's memory holds."""
    rng = np.random.default_rng(T)
    l, f = logits_of(rng, T, E)
    assert_routed(sg.route(l, k), f, k)


def test_route_ties_and_what_is_not_finite():
    inf, nan = float("inf"), float("nan")
    rows = [[1, 1, 1, 1, 1, 1], [0.0, -0.0, 0.0, -0.0, -1, 1], [-inf] * 6, [-inf, 2, -inf, -inf, -inf, -inf], [nan, 1, 2, 3, nan, 0],
            [inf, 1, inf, 0, 0, 0], [nan] * 6, [-inf, -inf, -inf, -inf, -inf, -3e38], [3e38, -3e38, 0, 1, 2, 3], [-200, -150, -300, -160, -170, -180],
            [-1e-45, 1e-45, 0, -0.0, 2e-45, -2e-45]]
    l = torch.tensor(rows, dtype=torch.float32, device="cuda")
    for k in (1, 3, 6):
        for how in HOW:
            got = sg.route(l, k, **how)
            e, w, offsets, order = oracle.route(l.double().cpu().numpy(), k, **how)
            assert np.array_equal(got.experts.cpu().numpy(), e), how
            assert np.array_equal(got.order.cpu().numpy(), order) and np.array_equal(got.offsets.cpu().numpy(), offsets)
            g = got.weights.double().cpu().numpy()
            # (exp of fp32 arguments: sigmoids near 0 underflow, and their quotients with them)
            near = [i for i in range(len(rows)) if i != 9]
            assert np.allclose(g[near], w[near], rtol=1e-5, atol=1e-30, equal_nan=True), how
            assert np.isfinite(g[9]).all()


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (33, 64, 6), (100, 300, 8), (20, 1024, 32), (9, 33, 33 - 1)])
def test_route_gradient(T, E, k, how):
    """Against the formula, and against differences of the fp64 oracle's weights."""
    rng = np.random.default_rng(T * 3 + E)
    for half in (False, True):
        l, f = logits_of(rng, T, E, half)
        l.requires_grad_(True)
        r = sg.route(l, k, **how)
        assert not r.experts.requires_grad and r.weights.requires_grad
        g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
        r.weights.backward(g)
        e = r.experts.cpu().numpy()
        gf = g.double().cpu().numpy()
        ref, S = oracle.route_backward(gf, f, e, **how)
        got = l.grad.double().cpu().numpy()
        assert l.grad.dtype == l.dtype
        bound = 4 * eps_of(E, f) * S + (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -10) if half else 0.0) + 2.0 ** -126
        assert (np.abs(got - ref) <= bound).all(), how
        assert torch.equal(l.grad, sg.route_backward(g, l.detach(), r.experts, **how))
        if half:
            continue
        # differences, of the choices held as they are
        step, t = 1e-5, int(rng.integers(T))
        for i in {int(e[t, 0]), int(rng.integers(E)), int(e[t, -1])}:
            def weights(d):
                x = f[t].copy()
                x[i] += d
                s = np.exp(x - x.max()) / np.exp(x - x.max()).sum() if how["score"] == "softmax" else 1 / (1 + np.exp(-x))
                p = s[e[t]]
                return how.get("factor", 1.0) * (p / p.sum() if how["renormalize"] else p)
            diff = float(gf[t] @ (weights(step) - weights(-step)) / (2 * step))
            assert abs(diff - got[t, i]) <= 1e-6 + 1e-4 * S[t, i], (how, i)


def test_route_gradient_of_masked_rows_and_bad_choices():
    inf = float("inf")
    l = torch.tensor([[-inf] * 4, [1, -inf, 2, -inf], [0, 1, 2, 3]], device="cuda")
    e = torch.tensor([[0, 1], [2, 0], [99, -5]], dtype=torch.int32, device="cuda")
    g = torch.tensor([[1.0, -2], [3, 1], [1, 1]], device="cuda")
    for how in HOW:
        d = sg.route_backward(g, l, e, **how)
        assert torch.isfinite(d).all() and not d[0].any() and not d[2].any()
        assert not d[1, 1].any() and not d[1, 3].any()
    d = sg.route_backward(g, l, e)   # two choices whose weights add up to one
    assert torch.allclose(d[1, 0], -d[1, 2], rtol=1e-5) and d[1, 2] > 0


def test_route_no_tokens_and_refusals():
    l = torch.zeros(0, 8, device="cuda")
    r = sg.route(l, 2)
    assert r.experts.shape == (0, 2) and r.order.shape == (0,) and not r.offsets.any()
    assert sg.route(l, 2, sort=False).weights.shape == (0, 2)
    assert sg.route_backward(r.weights, l, r.experts).shape == (0, 8)
    l = torch.zeros(3, 8, device="cuda")
    for bad, what in ((lambda: sg.route(l, 9), ValueError), (lambda: sg.route(l, 0), ValueError), (lambda: sg.route(l.half(), 2), TypeError),
                      (lambda: sg.route(l.t(), 2), ValueError), (lambda: sg.route(l, 2, score="relu"), ValueError),
                      (lambda: sg.route(l.cpu(), 2), TypeError), (lambda: sg.route(torch.zeros(2, 1025, device="cuda"), 2), ValueError),
                      (lambda: sg.route_backward(torch.zeros(3, 2, device="cuda"), l, torch.zeros(3, 2, device="cuda")), TypeError),
                      (lambda: sg.route_backward(torch.zeros(3, 2, device="cuda"), l, torch.zeros(2, 2, dtype=torch.int32, device="cuda")), ValueError)):
        with pytest.raises(what):
            bad()


# ---------------------------------------------------------------- whole layer


class Layer:
    def __init__(self, rng, E, H, I, fp8):
        w13, f13 = normal(rng, (E, 2 * I, H), H ** -0.5)
        w2, f2 = normal(rng, (E, H, I), I ** -0.5)
        self.fp8, self.E, self.H, self.I = fp8, E, H, I
        if fp8:
            self.W13, self.W2 = (sg.quantize_fp8(w, block_rows=128) for w in (w13, w2))
            self.values()
        else:
            self.W13, self.W2, self.f13, self.f2 = sg.GroupedWeight(w13), sg.GroupedWeight(w2), f13, f2

    def values(self):
        self.f13, self.f2 = (np.stack([oracle.fp8_values(c, s) for c, s in zip(*host(q))]) for q in (self.W13, self.W2))

    def status(self):
        return (sg.fp8_status if self.fp8 else sg.grouped_status)(self.W13)


def choices(rng, T, E, k):
    e = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    return torch.from_numpy(e).cuda(), torch.from_numpy(w).cuda(), e, w.astype(np.float64)


def assert_layer(got, Xf, layer, e, w, what=""):
    ref, B = oracle.moe_forward(Xf, layer.f13, layer.f2, e, w)
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bad = np.abs(got - ref) > 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * B
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:3])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 16, 16), (1, 8, 2, 1024, 528), (2, 3, 3, 272, 144), (5, 8, 1, 144, 1040), (8, 40, 6, 256, 272),
                                       (9, 8, 2, 528, 256), (13, 11, 3, 1008, 720), (16, 300, 4, 144, 48), (17, 5, 5, 272, 400),
                                       (33, 4, 2, 144, 272), (40, 64, 8, 128, 144), (64, 3, 3, 272, 144), (64, 40, 32, 48, 32)])
def test_moe(T, E, k, H, I, fp8):
    rng = np.random.default_rng(T * 11 + E)
    layer = Layer(rng, E, H, I, fp8)
    X, Xf = normal(rng, (T, H))
    e, w, ef, wf = choices(rng, T, E, k)
    Y = sg.moe_forward(X, layer.W13, layer.W2, e, w)
    assert_layer(Y, Xf, layer, ef, wf)
    out = torch.full_like(Y, float("nan"))
    assert sg.moe_forward(X, layer.W13, layer.W2, e, w, out=out) is out and torch.equal(out, Y)
    assert layer.status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(64, 1024, 32, 32, 48), (1, 1024, 32, 4112, 16)])
def test_moe_of_the_most_experts_tokens_and_choices(T, E, k, H, I, fp8):
    rng = np.random.default_rng(T * 11 + E)
    layer = Layer(rng, E, H, I, fp8)
    X, Xf = normal(rng, (T, H))
    e, w, ef, wf = choices(rng, T, E, k)
    Y = sg.moe_forward(X, layer.W13, layer.W2, e, w)
    assert_layer(Y, Xf, layer, ef, wf)
    out = torch.full_like(Y, float("nan"))
    assert sg.moe_forward(X, layer.W13, layer.W2, e, w, out=out) is out and torch.equal(out, Y)
    assert layer.status() == 0


@pytest.mark.parametrize("T,E,k,H,I", [(3, 5, 2, 1000, 712), (20, 4, 2, 8, 8), (64, 2, 1, 24, 40), (1, 2, 2, 712, 1000)])
def test_moe_multiples_of_eight(T, E, k, H, I):
    rng = np.random.default_rng(T)
    layer = Layer(rng, E, H, I, False)
    X, Xf = normal(rng, (T, H))
    e, w, ef, wf = choices(rng, T, E, k)
    assert_layer(sg.moe_forward(X, layer.W13, layer.W2, e, w), Xf, layer, ef, wf)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 8, 12, 33, 64])
def test_moe_one_expert_for_all_twice_chosen_and_bad_choices(T, fp8):
    rng = np.random.default_rng(T)
    layer = Layer(rng, 6, 272, 144, fp8)
    X, Xf = normal(rng, (T, 272))
    e = np.full((T, 3), 4, dtype=np.int32)      # one expert, three times
    w = rng.standard_normal((T, 3)).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()
    got = sg.moe_forward(X, layer.W13, layer.W2, dev(e), dev(w))
    total = (w[:, 0] + w[:, 1] + w[:, 2])[:, None]
    assert_layer(got, Xf, layer, e[:, :1], total.astype(np.float64), "one expert")
    assert layer.status() == 0
    e[:, 1], e[:, 2] = 2 ** 30, -1              # out of range: count for nothing
    got = sg.moe_forward(X, layer.W13, layer.W2, dev(e), dev(w))
    assert layer.status() == 1 and layer.status() == 0
    assert_layer(got, Xf, layer, e[:, :1], w[:, :1].astype(np.float64), "bad choices")
    e[:] = 6
    assert not sg.moe_forward(X, layer.W13, layer.W2, dev(e), dev(w)).any()
    assert layer.status() == 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [4, 14, 40])
def test_moe_nan_stays_where_it_belongs(T, fp8):
    """A token's NaN reaches its own row; an expert's reaches its own tokens, and nobody when it is not chosen."""
    rng = np.random.default_rng(T)
    layer = Layer(rng, 5, 272, 144, fp8)
    X, Xf = normal(rng, (T, 272))
    ef = np.stack([rng.permutation(3)[:2] for _ in range(T)]).astype(np.int32)   # experts 0 .. 2
    ef[T // 2] = [3, 0]
    w = rng.random((T, 2)).astype(np.float32)
    e, wd = torch.from_numpy(ef).cuda(), torch.from_numpy(w).cuda()
    clean = sg.moe_forward(X, layer.W13, layer.W2, e, wd)

    def poison(W, at):
        if fp8:
            W.codes.view(torch.uint8)[at] = 0x7F
        else:
            W.weight[at] = float("nan")

    poison(layer.W13, 4)          # nobody's
    poison(layer.W2, 4)
    assert torch.equal(sg.moe_forward(X, layer.W13, layer.W2, e, wd), clean)
    X2 = X.clone()
    X2[1, 5] = float("nan")
    got = sg.moe_forward(X2, layer.W13, layer.W2, e, wd)
    rest = torch.arange(T, device="cuda") != 1
    assert torch.isnan(got[1]).all() and torch.equal(got[rest], clean[rest])
    poison(layer.W13, (3, 200, 17))   # expert 3's up row 56: NaN in h, and in all of its token's outputs
    got = sg.moe_forward(X, layer.W13, layer.W2, e, wd)
    rest = torch.arange(T, device="cuda") != T // 2
    assert torch.isnan(got[T // 2]).all() and torch.equal(got[rest], clean[rest])
    layer = Layer(np.random.default_rng(T), 5, 272, 144, fp8)
    poison(layer.W2, (3, 37, 143))    # output feature 37
    got = sg.moe_forward(X, layer.W13, layer.W2, e, wd)
    assert torch.isnan(got[T // 2, 37]) and int(torch.isnan(got).sum()) == 1
    got[T // 2, 37] = clean[T // 2, 37]
    assert torch.equal(got, clean)


def test_moe_of_every_code():
    """Each finite e4m3 code in both weights, at scales far from one."""
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    rng = np.random.default_rng(3)
    layer = Layer(rng, 2, 256, 272, True)
    for q, scale in ((layer.W13, 1e-4), (layer.W2, 1e-3)):
        pick = rng.choice(codes, q.shape).astype(np.uint8)
        q.codes.view(torch.uint8).copy_(torch.from_numpy(pick))
        q.scales.copy_(torch.from_numpy((scale * rng.random(tuple(q.scales.shape))).astype(np.float32)))
    layer.values()
    X, Xf = normal(rng, (9, 256))
    e, w, ef, wf = choices(rng, 9, 2, 1)
    assert_layer(sg.moe_forward(X, layer.W13, layer.W2, e, w), Xf, layer, ef, wf)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 11, 50])
def test_router_and_layer_together(T, fp8):
    """Router and layer in one stream, eager and as a replayed graph; and the same layer through the sorted pairs and
    the grouped products."""
    rng = np.random.default_rng(T)
    E, k, H, I = 16, 4, 272, 144
    layer = Layer(rng, E, H, I, fp8)
    layer.W13.status, layer.W2.status
    X, Xf = normal(rng, (T, H))
    l, lf = logits_of(rng, T, E)
    r = sg.route(l, k)
    Y = sg.moe_forward(X, layer.W13, layer.W2, r.experts, r.weights)
    e, w = r.experts.cpu().numpy(), r.weights.double().cpu().numpy()
    assert_layer(Y, Xf, layer, e, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rg = sg.route(l, k, sort=False)
        Yg = sg.moe_forward(X, layer.W13, layer.W2, rg.experts, rg.weights)
    for rep in range(4):
        l.copy_(logits_of(rng, T, E)[0])
        X.copy_(normal(rng, (T, H))[0])
        g.replay()
        torch.cuda.synchronize()
        rr = sg.route(l, k)
        assert torch.equal(Yg, sg.moe_forward(X, layer.W13, layer.W2, rr.experts, rr.weights))
    # sorted rows through the grouped products: rounded once more per product, so only near
    if fp8:
        return
    r, Y = rr, Yg
    rows = X[r.order // k]
    gate, up = sg.grouped_forward(rows, layer.W13, r.offsets).float().chunk(2, dim=1)
    h = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
    y = sg.grouped_forward(h, layer.W2, r.offsets).float() * r.weights.flatten()[r.order.long(), None]
    out = torch.zeros(T, H, device="cuda").index_add_(0, r.order.long() // k, y)
    assert (out - Y.float()).abs().max() <= 0.05 * Y.float().abs().max()


def test_moe_back_to_back_without_waits():
    """Calls that feed one another over two buffers, with router, eager without waits and with one behind each."""
    rng = np.random.default_rng(5)
    E, k, H, I, T = 12, 3, 256, 272, 9
    layers = [Layer(rng, E, H, I, i % 2 == 1) for i in range(4)]
    X, _ = normal(rng, (T, H))
    ls = [logits_of(rng, T, E)[0] for _ in range(8)]

    def chain(wait):
        out = []
        for start in range(6):   # three layers deep: each about squares its input, eight would underflow to zeros
            A, B = X.clone(), torch.empty_like(X)
            for i in range(start, start + 3):
                r = sg.route(ls[i], k, sort=False)
                wait()
                sg.moe_forward(A, layers[i % 4].W13, layers[i % 4].W2, r.experts, r.weights, out=B)
                wait()
                A, B = B, A
            out.append(A)
        return torch.stack(out)

    want = chain(torch.cuda.synchronize)
    assert torch.isfinite(want.float()).all() and want.any()
    for _ in range(5):
        assert torch.equal(chain(lambda: None), want)


def test_moe_weights_made_just_before():
    """Weights written by the kernel before the layer's call are those it multiplies, down weights too."""
    rng = np.random.default_rng(6)
    E, H, I, T = 3, 512, 528, 4
    banks = [(normal(rng, (E, 2 * I, H), 0.05)[0], normal(rng, (E, H, I), 0.05)[0]) for _ in range(3)]
    q13, q2 = (sg.quantize_fp8(w, block_rows=128) for w in banks[0])
    X, _ = normal(rng, (T, H))
    e, w, _, _ = choices(rng, T, E, 2)
    want = []
    for b13, b2 in banks:
        want.append(sg.moe_forward(X, sg.quantize_fp8(b13, block_rows=128), sg.quantize_fp8(b2, block_rows=128), e, w))
        torch.cuda.synchronize()
    for rep in range(10):
        got = []
        for b13, b2 in banks:
            sg.quantize_fp8(b13, block_rows=128, out=q13)
            sg.quantize_fp8(b2, block_rows=128, out=q2)
            got.append(sg.moe_forward(X, q13, q2, e, w))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_moe_no_tokens_and_refusals():
    rng = np.random.default_rng(7)
    layer, layer8 = Layer(rng, 2, 48, 32, False), Layer(rng, 2, 48, 32, True)
    X, _ = normal(rng, (4, 48))
    e, w, _, _ = choices(rng, 4, 2, 2)
    assert sg.moe_forward(X[:0], layer.W13, layer.W2, e[:0], w[:0]).shape == (0, 48)
    big = torch.zeros(65, 48, dtype=torch.bfloat16, device="cuda")
    for bad, what in ((lambda: sg.moe_forward(big, layer.W13, layer.W2, e, w), ValueError),
                      (lambda: sg.moe_forward(X, layer.W13, layer8.W2, e, w), TypeError),
                      (lambda: sg.moe_forward(X, layer.W2, layer.W13, e, w), ValueError),
                      (lambda: sg.moe_forward(X[:, :32].contiguous(), layer.W13, layer.W2, e, w), ValueError),
                      (lambda: sg.moe_forward(X, layer.W13, layer.W2, e.long(), w), TypeError),
                      (lambda: sg.moe_forward(X, layer.W13, layer.W2, e, w.double()), TypeError),
                      (lambda: sg.moe_forward(X, layer.W13, layer.W2, e[:3], w), ValueError),
                      (lambda: sg.moe_forward(X, layer.W13, layer.W2, e, w[:, :1].contiguous()), ValueError),
                      (lambda: sg.moe_forward(X, layer.W13, layer.W2, e, w, out=X), ValueError),
                      (lambda: sg.moe_forward(X, layer.W13, layer.W2, torch.zeros(4, 33, dtype=torch.int32, device="cuda"),
                                              torch.zeros(4, 33, device="cuda")), ValueError)):
        with pytest.raises(what):
            bad()
