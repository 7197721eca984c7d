"""Sigmoid weights that are divided by their sum, of logits far below zero, where the sigmoids are no fp32 numbers and their
quotients are: against the quotients in 64 bits, taken in logarithms, and their gradient against the formula and against
differences.

Bound: an exponential is off by 2^-22 and by 2^-24 of its argument, a rounded difference; a score has two of them, a sum and a
division, a weight the sum of up to 32 scores, a division and a product.  A gradient has two such weights and some products and
differences, of which S below sums the absolute terms."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def log_sigmoid(l):
    return np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))


def weights(l, e):
    """Quotients [T, k] of the chosen sigmoids in 64 bits."""
    s = log_sigmoid(np.take_along_axis(l, e, 1))
    s = np.exp(s - s.max(1, keepdims=True))
    return s / s.sum(1, keepdims=True)


def eps(l, e):
    chosen = np.take_along_axis(l, e, 1)
    spread = (chosen.max(1) - chosen.min(1))[:, None]
    return 2 * (2 * 2.0 ** -22 + spread * 2.0 ** -24 + 3 * 2.0 ** -24) + (5 + 3) * 2.0 ** -24


def check(l, k, factor=1.0):
    T, E = l.shape
    rng = np.random.default_rng(T)
    g = rng.standard_normal((T, k)).astype(np.float32)
    t = torch.from_numpy(l.astype(np.float32)).cuda().requires_grad_(True)
    l = t.detach().double().cpu().numpy()
    r = sg.route(t, k, score="sigmoid", factor=factor)
    e = r.experts.long().cpu().numpy()
    assert np.array_equal(e, np.argsort(-l, axis=1, kind="stable")[:, :k])
    w = weights(l, e)
    got = r.weights.detach().double().cpu().numpy() / factor
    assert (np.abs(got - w) <= eps(l, e) * w + 2.0 ** -126).all(), np.abs(got - w).max()
    r.weights.backward(torch.from_numpy(g).cuda())
    # dw_i / dl_j = w_i (1[i = j] - w_j) (1 - sigmoid(l_j))
    g = g.astype(np.float64)
    slope = factor * w / (1 + np.exp(np.take_along_axis(l, e, 1)))
    want, S = slope * (g - (g * w).sum(1, keepdims=True)), slope * (np.abs(g) + np.abs(g * w).sum(1, keepdims=True))
    grad = t.grad.double().cpu().numpy()
    chosen = np.take_along_axis(grad, e, 1)
    assert (np.abs(chosen - want) <= 4 * eps(l, e) * S + 2.0 ** -126).all(), np.abs(chosen - want).max()
    np.put_along_axis(grad, e, 0, 1)
    assert not grad.any()
    # differences along the gradient of one chosen logit, the choices held
    step = 1e-5
    for j in {0, k - 1}:
        up, down = l.copy(), l.copy()
        np.put_along_axis(up, e[:, j:j + 1], np.take_along_axis(l, e[:, j:j + 1], 1) + step, 1)
        np.put_along_axis(down, e[:, j:j + 1], np.take_along_axis(l, e[:, j:j + 1], 1) - step, 1)
        diff = factor * (g * (weights(up, e) - weights(down, e))).sum(1) / (2 * step)
        assert (np.abs(diff - chosen[:, j]) <= 1e-6 + 1e-4 * S[:, j]).all()


@pytest.mark.parametrize("rows", [[-90, -91, -92, -93], [-150, -160, -170, -200], [-86.5, -87.5, -88.5, -89.5], [-100, -101.5, -103, -104.5],
                                  [-699, -699.5, -699.25, -800], [-300] * 4, [0, -100, -50, -120], [-16, -100, -95, -90], [5, -95, 2, -100],
                                  [-32, -88, -89, -110], [40, -40, -100, 100], [-1e-3, 1e-3, -90, -90]])
@pytest.mark.parametrize("k", [1, 2, 4])
def test_rows_far_below_zero(rows, k):
    check(np.array([rows, rows[::-1]], dtype=np.float64), k)


@pytest.mark.parametrize("T,E,k,low,high", [(200, 40, 6, -600, 5), (64, 8, 8, -100, -80), (130, 300, 32, -200, -85), (33, 1024, 8, -690, -500),
                                            (500, 64, 6, -40, 0)])
def test_many_rows(T, E, k, low, high):
    rng = np.random.default_rng(E)
    check(rng.uniform(low, high, (T, E)), k, factor=2.5)


def test_rows_of_nothing():
    """Nothing above -700: weights and gradients of zero, as in a row of -inf; half-precision masks of the lowest value too."""
    inf = float("inf")
    l = torch.tensor([[-701.0, -702, -800, -inf], [-3e38, -3e38, -inf, -inf], [-inf] * 4, [-1e9, -1e9, -1e9, -750]], device="cuda")
    for logits in (l, l.to(torch.bfloat16), torch.full((3, 4), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16, device="cuda")):
        r = sg.route(logits, 2, score="sigmoid")
        low = logits.float().amax(1) < -700   # (bf16 has -700 and -704, so that -701 becomes -700)
        assert not r.weights[low].any() and low.sum() >= 3
        g = torch.ones(logits.shape[0], 2, device="cuda")
        assert not sg.route_backward(g, logits, r.experts, score="sigmoid")[low].any()
        for t in torch.nonzero(~low).flatten().tolist():
            l64, e = logits[t:t + 1].double().cpu().numpy(), r.experts[t:t + 1].long().cpu().numpy()
            assert np.allclose(r.weights[t].cpu().numpy(), weights(l64, e)[0], rtol=1e-6)


def test_a_masked_choice_beside_a_low_one():
    l = torch.tensor([[-120.0, -float("inf"), -121.0, -float("inf")]], device="cuda")
    r = sg.route(l, 4, score="sigmoid")
    want = 1 / (1 + np.exp(-1.0))
    assert np.allclose(r.weights.cpu().numpy(), [[want, 1 - want, 0, 0]], rtol=1e-6)
    d = sg.route_backward(torch.tensor([[1.0, 0, 5, 7]], device="cuda"), l, r.experts, score="sigmoid").cpu().numpy()
    assert np.allclose(d, [[want * (1 - want), 0, -want * (1 - want), 0]], rtol=1e-5)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("E,k", [(6, 2), (40, 8), (300, 32)])
def test_a_nan_that_was_not_chosen(E, k, renormalize):
    """It changes no sigmoid weight, and no gradient but its own, which is zero."""
    rng = np.random.default_rng(E)
    l = torch.from_numpy(rng.standard_normal((20, E)).astype(np.float32)).cuda()
    g = torch.from_numpy(rng.standard_normal((20, k)).astype(np.float32)).cuda()
    how = dict(score="sigmoid", renormalize=renormalize)
    r = sg.route(l, k, **how)
    want = sg.route_backward(g, l, r.experts, **how)
    last = l.argmin(1, keepdim=True)
    bad = l.scatter(1, last, float("nan"))
    got = sg.route(bad, k, **how)
    assert torch.equal(got.experts, r.experts) and torch.equal(got.weights, r.weights)
    d = sg.route_backward(g, bad, got.experts, **how)
    assert torch.equal(d, want) and not d.gather(1, last).any()


@pytest.mark.parametrize("how", [dict(), dict(renormalize=False, factor=2.5), dict(score="sigmoid")])
def test_gradient_without_sorting(how):
    """route(sort=False) has no offsets and no order, and the same gradient."""
    rng = np.random.default_rng(7)
    l = torch.from_numpy(rng.standard_normal((300, 40)).astype(np.float32)).cuda()
    g = torch.from_numpy(rng.standard_normal((300, 4)).astype(np.float32)).cuda()
    grads = []
    for sort in (False, True):
        t = l.clone().requires_grad_(True)
        r = sg.route(t, 4, sort=sort, **how)
        assert (r.offsets is None) == (r.order is None) == (not sort) and r.weights.requires_grad
        r.weights.backward(g)
        grads.append(t.grad)
    assert torch.equal(*grads) and torch.equal(grads[0], sg.route_backward(g, l, r.experts, **how))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [1, 2, 33, 256, 1024])
def test_an_only_choice_that_is_divided_by_itself(E, score):
    """Its weight is the factor, whatever the logits, and their gradient is zero, not a rounding."""
    rng = np.random.default_rng(E)
    for half in (False, True):
        l = torch.from_numpy((rng.standard_normal((500, E)) * 3 - 2).astype(np.float32)).cuda()
        l = l.to(torch.bfloat16) if half else l
        g = torch.from_numpy(rng.standard_normal((500, 1)).astype(np.float32)).cuda()
        r = sg.route(l, 1, score=score, factor=0.7)
        assert (r.weights == np.float32(0.7)).all()
        assert not sg.route_backward(g, l, r.experts, score=score, factor=0.7).any()
