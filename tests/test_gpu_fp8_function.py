"""Autograd of the 8-bit layer: the bias's gradient, weights that change between forward and backward, ranks of the weight
and the offsets."""
import numpy as np
import pytest
import torch

from oracle import experts
from tests._experts import check, normal, offsets_of
from tests.test_gpu_fp8 import weights

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


@pytest.mark.parametrize("rows,N", [([1], 24), ([700], 144), ([5, 0, 70, 33], 144), ([3, 0, 300], 136)])
@pytest.mark.parametrize("with_input", [False, True])
def test_gradient_of_a_trained_bias(rows, N, with_input):
    """Column sums of the upstream gradient, over an expert's rows; with and without the input's gradient beside it (which
    wants output features in sixteens)."""
    if with_input and N % 16:
        N = 144
    rng = np.random.default_rng(sum(rows) + N)
    front = 0 if len(rows) == 1 else 2
    off, o = offsets_of(rows, front)
    T, E = sum(rows) + 2 * front, len(rows)
    Wq, _ = weights(rng, *((N, 272) if E == 1 else (E, N, 272)))
    X, _ = normal(rng, (T, 272))
    bias, _ = normal(rng, (N,) if E == 1 else (E, N))
    X.requires_grad_(with_input)
    bias.requires_grad_(True)
    Y = sg.Fp8LinearFunction.apply(X, Wq, None if E == 1 else off, bias)
    g, gf = normal(rng, (T, N))
    Y.backward(g)
    ref, S = experts.grouped_bias_grad(gf, o)
    check(bias.grad.view(E, N), ref, S, max(rows), "bias")
    if with_input:
        call = sg.backward_input_fp8(g, Wq) if E == 1 else sg.grouped_backward_input_fp8(g, Wq, off)
        assert torch.equal(X.grad, call)
    else:
        assert X.grad is None
    # differences: the sum of Y times g is linear in the bias
    step = torch.zeros_like(bias)
    step.view(-1)[5] = 1.0
    with torch.no_grad():
        more = sg.Fp8LinearFunction.apply(X, Wq, None if E == 1 else off, (bias * 0 + step))
        none = sg.Fp8LinearFunction.apply(X, Wq, None if E == 1 else off, (bias * 0))
    diff = ((more.double() - none.double()) * g.double()).sum()
    size = ((more.double().abs() + none.double().abs()) * g.double().abs() * (more != none)).sum()
    assert (diff - bias.grad.view(-1)[5].double()).abs() <= 2.0 ** -8 * (size + bias.grad.view(-1)[5].double().abs())


def test_gradient_of_a_trained_bias_of_broadcast_and_no_rows():
    rng = np.random.default_rng(1)
    Wq, _ = weights(rng, 144, 272)
    bias = torch.zeros(144, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    X, _ = normal(rng, (9, 272))
    sg.Fp8LinearFunction.apply(X, Wq, None, bias).sum().backward()
    assert (bias.grad == 9).all()
    bias.grad = None
    sg.Fp8LinearFunction.apply(X[:0], Wq, None, bias).sum().backward()
    assert not bias.grad.any()


def test_arguments_that_are_left_out():
    rng = np.random.default_rng(5)
    Wq, _ = weights(rng, 2, 144, 272)
    one = sg.Fp8Tensor(Wq.codes[0], Wq.scales[0])
    off, _ = offsets_of([4, 5])
    X, _ = normal(rng, (9, 272))
    X.requires_grad_(True)
    g, _ = normal(rng, (9, 144))
    for args, want in (((one,), lambda: sg.backward_input_fp8(g, one)), ((one, None), lambda: sg.backward_input_fp8(g, one)),
                       ((Wq, off), lambda: sg.grouped_backward_input_fp8(g, Wq, off))):
        got, = torch.autograd.grad(sg.Fp8LinearFunction.apply(X, *args), X, g)
        assert torch.equal(got, want())


def test_a_trained_bias_in_a_captured_backward():
    rng = np.random.default_rng(2)
    Wq, _ = weights(rng, 144, 272)
    Wq.status
    X, _ = normal(rng, (70, 272))
    bias, _ = normal(rng, (144,))
    bias.requires_grad_(True)
    g, _ = normal(rng, (70, 144))
    want, = torch.autograd.grad(sg.Fp8LinearFunction.apply(X, Wq, None, bias), bias, g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(sg.Fp8LinearFunction.apply(X, Wq, None, bias), bias, g)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("grouped", [False, True])
def test_a_weight_that_changed_before_the_backward_is_refused(grouped):
    rng = np.random.default_rng(3)
    shape = (2, 144, 272) if grouped else (144, 272)
    W, _ = normal(rng, shape)
    other, _ = normal(rng, shape)
    off, _ = offsets_of([4, 5])
    make = sg.GroupedFp8Linear if grouped else sg.Fp8Linear
    args = (off,) if grouped else ()
    x, _ = normal(rng, (9, 272))
    x.requires_grad_(True)
    g, _ = normal(rng, (9, 144))
    for change in (lambda m: sg.quantize_fp8(other, block_rows=128, out=m.weight8), lambda m: m.load_state_dict(make.from_dense(other).state_dict()),
                   lambda m: m.scales.add_(1), lambda m: m.codes.zero_()):
        layer = make.from_dense(W)
        y = layer(x, *args)
        change(layer)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward(g)
        layer(x, *args).backward(g)   # the changed weight, once it is the forward's too
        assert torch.isfinite(x.grad.float()).all()
        x.grad = None


def test_weights_of_inference_mode_and_two_backwards():
    """Inference tensors have no versions and are used as they are; an unchanged weight may be gone through twice."""
    rng = np.random.default_rng(4)
    W, _ = normal(rng, (144, 272))
    with torch.inference_mode():
        Wi = sg.quantize_fp8(W, block_rows=128)
    Wq = sg.quantize_fp8(W, block_rows=128)
    x, _ = normal(rng, (9, 272))
    x.requires_grad_(True)
    g, _ = normal(rng, (9, 144))
    want = sg.backward_input_fp8(g, Wq)
    for w in (Wi, Wq):
        y = sg.Fp8LinearFunction.apply(x, w)
        for _ in range(2):
            got, = torch.autograd.grad(y, x, g, retain_graph=True)
            assert torch.equal(got, want)
    with torch.inference_mode():
        sg.quantize_fp8(W, block_rows=128, out=Wi)
        sg.quantize_fp8(W, block_rows=128, out=Wq)
        assert torch.equal(sg.Fp8LinearFunction.apply(x, Wq), y)


def test_offsets_go_with_weights_of_experts_only():
    """A weight [N, K] with offsets, which would be left aside, and weights [E, N, K] without are refused."""
    rng = np.random.default_rng(6)
    Wq, _ = weights(rng, 2, 144, 272)
    one = sg.Fp8Tensor(Wq.codes[0], Wq.scales[0])
    off, _ = offsets_of([4, 5])
    X, _ = normal(rng, (9, 272))
    for bad in (lambda: sg.Fp8LinearFunction.apply(X, one, off), lambda: sg.Fp8LinearFunction.apply(X, Wq),
                lambda: sg.GroupedFp8Linear(one)(X, off), lambda: sg.Fp8Linear(Wq)(X), lambda: sg.GroupedFp8Linear(Wq)(X, None)):
        with pytest.raises(ValueError, match="Wq must be an Fp8Tensor"):
            bad()
    assert torch.equal(sg.GroupedFp8Linear(Wq)(X, off), sg.grouped_forward_fp8(X, Wq, off))
