"""Rows, gradients and weights that begin on any element: views into flat buffers, as a concatenation
or an optimizer's flat storage hands them on."""
import numpy as np
import pytest
import torch

from tests._experts import integers, normal, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def shifted(t, by):
    """A copy of t that begins `by` elements into a buffer."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device=t.device)
    view = flat[by:].view(t.shape)
    view.copy_(t.detach())
    return view


@pytest.mark.parametrize("by", [1, 3, 8])
@pytest.mark.parametrize("rows", [[3, 0, 2], [70, 0, 50]])
def test_expert_layer(rows, by):
    rng = np.random.default_rng(51)
    off, T, N, K = offsets_of(rows)[0], sum(rows), 72, 40
    W, b, X, dY = (integers(rng, s)[0] for s in ((3, N, K), (3, N), (T, K), (T, N)))
    plain = sg.GroupedLinear(W.clone(), b.clone())
    x = X.clone().requires_grad_(True)
    y = plain(x, off)
    y.backward(dY)
    layer = sg.GroupedLinear(shifted(W, by), shifted(b, by))
    xs = shifted(X, by).requires_grad_(True)
    ys = layer(xs, off)
    assert torch.equal(ys, y)
    head = torch.ones(by, dtype=torch.bfloat16, device="cuda")
    w = torch.cat([head, dY.flatten()])
    (torch.cat([head, ys.flatten()]) * w).sum().backward()          # the gradient is a view at `by`
    assert torch.equal(xs.grad, x.grad)
    assert torch.equal(layer.weight.grad, plain.weight.grad) and torch.equal(layer.bias.grad, plain.bias.grad)
    ys = layer(xs.detach()[:, :], off)
    assert torch.equal(ys, y)


@pytest.mark.parametrize("by", [1, 3, 8])
@pytest.mark.parametrize("T", [2, 60])
def test_4_bit_layers(T, by):
    rng = np.random.default_rng(52)
    W, b, X = (normal(rng, s)[0] for s in ((72, 96), (72,), (T, 96)))
    want = sg.Mx4Linear.from_dense(W, b)(X)
    assert torch.equal(sg.Mx4Linear.from_dense(shifted(W, by), shifted(b, by))(shifted(X, by)), want)
    W3, b3, off = W.expand(2, 72, 96).contiguous(), b.expand(2, 72).contiguous(), offsets_of([1, T - 1])[0]
    assert torch.equal(sg.GroupedMx4Linear.from_dense(shifted(W3, by), shifted(b3, by))(shifted(X, by), off), want)


def test_calls_that_take_what_they_are_given_refuse():
    X, W, dY = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((4, 64), (2, 32, 64), (4, 32)))
    off = offsets_of([2, 2])[0]
    Wg, Wq = sg.GroupedWeight(W), sg.quantize_mx4(W)
    for call in (lambda: sg.grouped_forward(shifted(X, 1), Wg, off), lambda: sg.grouped_forward(X, Wg, off, out=shifted(dY, 1)),
                 lambda: sg.grouped_forward(X, sg.GroupedWeight(shifted(W, 1)), off),
                 lambda: sg.grouped_backward_input(shifted(dY, 1), Wg, off),
                 lambda: sg.grouped_backward_weight(dY, shifted(X, 1), Wg, off),
                 lambda: sg.grouped_bias_grad(shifted(dY, 1), off), lambda: sg.quantize_mx4(shifted(X, 1)),
                 lambda: sg.grouped_forward_mx4(shifted(X, 1), Wq, off)):
        with pytest.raises(sg.BslError):
            call()
    assert sg.grouped_status(Wg) == 0 and sg.mx4_status(Wq) == 0
