"""GPU parity of the expert (grouped) layer against the fp64 oracle: forward,
input, weight and bias gradient, through the binding and through autograd."""
import numpy as np
import pytest
import torch

from oracle import experts
from tests._experts import check, integers, normal, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def run_all(rows, N, K, seed, *, bias=True, first=0, spare=0, make=normal):
    rng = np.random.default_rng(seed)
    E, T = len(rows), first + sum(rows) + spare
    off, o = offsets_of(rows, first)
    X, Xf = make(rng, (T, K))
    W, Wf = make(rng, (E, N, K))
    dY, dYf = make(rng, (T, N))
    b, bf = make(rng, (E, N)) if bias else (None, None)
    Wg = sg.GroupedWeight(W)
    Y = sg.grouped_forward(X, Wg, off, bias=b)
    dX = sg.grouped_backward_input(dY, Wg, off)
    dW = sg.grouped_backward_weight(dY, X, Wg, off)
    db = sg.grouped_bias_grad(dY, off)
    torch.cuda.synchronize()
    assert sg.grouped_status(Wg) == 0
    depth = np.asarray(rows, dtype=float)
    return [(Y, *experts.grouped_forward(Xf, Wf, o, bf), K, "Y"),
            (dX, *experts.grouped_backward_input(dYf, Wf, o), N, "dX"),
            (dW, *experts.grouped_backward_weight(dYf, Xf, o), depth[:, None, None], "dW"),
            (db, *experts.grouped_bias_grad(dYf, o), 16 * depth[:, None], "db")]


CASES = [
    # rows of the experts, N, K, rows before the first and behind the last expert
    ([1], 8, 8, 0, 0),
    ([0, 1, 0], 8, 64, 0, 0),
    ([3, 0, 2], 64, 72, 2, 3),
    ([1, 1, 1, 1, 1, 1, 1, 1], 264, 136, 0, 0),
    ([16, 17, 15, 0, 31, 33], 136, 200, 0, 5),
    ([63, 64, 65, 127, 128, 129], 128, 64, 1, 0),
    ([255, 256, 257, 0], 256, 128, 0, 0),
    ([300, 5, 0, 700], 520, 1000, 0, 37),
    ([513], 1032, 776, 3, 9),
    ([2, 0, 0, 90], 2056, 320, 0, 0),
    ([40, 600], 72, 2048, 0, 0),
    ([0, 0, 0], 64, 64, 4, 4),
]


@pytest.mark.parametrize("rows,N,K,first,spare", CASES)
def test_parity(rows, N, K, first, spare):
    for got, ref, S, depth, what in run_all(rows, N, K, 11, first=first, spare=spare, bias=spare % 2 == 1):
        check(got, ref, S, depth, what)


@pytest.mark.parametrize("E,N,K", [(70, 64, 64), (1024, 16, 24)])
def test_many_experts(E, N, K):
    rows = np.random.default_rng(E).integers(0, 4, E).tolist()
    for got, ref, S, depth, what in run_all(rows, N, K, 12):
        check(got, ref, S, depth, what)


FEW = [([8], 1032, 4096, 0, 0), ([7], 24, 1000, 0, 0), ([0, 3, 0, 0, 1, 0, 2], 520, 2056, 1, 1), ([1] * 8, 264, 40, 0, 0),
       ([0] * 31 + [2] + [0] * 200 + [1, 0, 3], 72, 136, 0, 2), ([0] * 1000 + [5], 16, 264, 2, 1), ([9], 136, 1000, 0, 0),
       ([3, 0, 11], 264, 1000, 1, 1), ([16], 1032, 520, 0, 0), ([20, 1, 0, 8], 72, 2056, 2, 1), ([32], 4096, 2048, 0, 0),
       ([17], 8200, 4096, 0, 0), ([33], 136, 520, 0, 0)]


@pytest.mark.parametrize("rows,N,K,first,spare", FEW)
def test_few_rows(rows, N, K, first, spare):
    """Few rows in all, on both sides of 8, 16 and 32 and of the weights' sizes: any expert, long and odd K."""
    for got, ref, S, depth, what in run_all(rows, N, K, 20, first=first, spare=spare):
        check(got, ref, S, depth, what)


@pytest.mark.parametrize("rows,N,K", [([130, 0, 70, 1], 264, 520), ([2, 3], 72, 264), ([600, 20], 40, 1032)])
def test_exact_on_integers(rows, N, K):
    """Sums of small integers are exact in fp32: one rounding to bf16 remains."""
    for got, ref, _, _, what in run_all(rows, N, K, 13, make=integers):
        assert torch.equal(got.cpu(), torch.from_numpy(ref).float().to(torch.bfloat16)), what


@pytest.mark.parametrize("T,N,K", [(40, 264, 192), (700, 136, 320)])
@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_other_experts_rows_do_not_leak(T, N, K, junk):
    """NaN or infinities in one expert's rows and in the rows of none reach no other expert's outputs."""
    rng = np.random.default_rng(14)
    rows = [T // 4, T // 4 + 3, 1, T // 2 - 9]
    off, o = offsets_of(rows, 2)
    total = int(o[-1]) + 6
    X, _ = normal(rng, (total, K))
    dY, _ = normal(rng, (total, N))
    Wg = sg.GroupedWeight(normal(rng, (4, N, K))[0])
    clean = (sg.grouped_forward(X, Wg, off), sg.grouped_backward_input(dY, Wg, off),
             sg.grouped_backward_weight(dY, X, Wg, off), sg.grouped_bias_grad(dY, off))
    bad = torch.ones(total, dtype=torch.bool)
    bad[int(o[0]):int(o[1])] = False
    bad[int(o[2]):int(o[4])] = False          # expert 1 and the rows of none stay bad
    X2, dY2 = X.clone(), dY.clone()
    X2[bad.cuda()] = junk
    dY2[bad.cuda()] = junk
    dirty = (sg.grouped_forward(X2, Wg, off), sg.grouped_backward_input(dY2, Wg, off),
             sg.grouped_backward_weight(dY2, X2, Wg, off), sg.grouped_bias_grad(dY2, off))
    good = (~bad).cuda()
    for a, b in zip(clean[:2], dirty[:2]):
        assert torch.equal(a[good], b[good])
        assert not b[:2].any() and not b[int(o[4]):].any()     # rows of none: zeros
    for a, b in zip(clean[2:], dirty[2:]):
        for e in (0, 2, 3):
            assert torch.equal(a[e], b[e])
        assert not torch.isfinite(b[1].float()).any()


@pytest.mark.parametrize("rows,N,K", [([5, 0, 9], 72, 64), ([300, 0, 200], 264, 136)])
def test_rows_of_no_expert_stay_in_out(rows, N, K):
    rng = np.random.default_rng(15)
    off, o = offsets_of(rows, 3)
    T = int(o[-1]) + 7
    X, _ = normal(rng, (T, K))
    dY, _ = normal(rng, (T, N))
    Wg = sg.GroupedWeight(normal(rng, (3, N, K))[0])
    for fn, a, cols in ((sg.grouped_forward, X, N), (sg.grouped_backward_input, dY, K)):
        want = fn(a, Wg, off)
        frame = torch.full((T + 4, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        out = frame[2:T + 2]
        assert fn(a, Wg, off, out=out) is out
        assert torch.equal(out[int(o[0]):int(o[-1])], want[int(o[0]):int(o[-1])])
        rest = torch.cat([frame[:2 + int(o[0])], frame[2 + int(o[-1]):]])
        assert (rest == 7.0).all()
        assert not want[:int(o[0])].any() and not want[int(o[-1]):].any()


def test_weight_gradient_writes_nothing_else():
    rng = np.random.default_rng(16)
    off, _ = offsets_of([70, 0, 3])
    N, K = 264, 72
    X, _ = normal(rng, (73, K))
    dY, _ = normal(rng, (73, N))
    Wg = sg.GroupedWeight(normal(rng, (3, N, K))[0])
    frame = torch.full((5, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    out = sg.grouped_backward_weight(dY, X, Wg, off, out=frame[1:4])
    assert torch.equal(out, sg.grouped_backward_weight(dY, X, Wg, off))
    assert (frame[0] == 7.0).all() and (frame[4] == 7.0).all()
    assert not out[1].any()


def test_no_rows_at_all():
    N, K = 64, 72
    Wg = sg.GroupedWeight(torch.ones(2, N, K, dtype=torch.bfloat16, device="cuda"))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    X, dY = (torch.empty(0, c, dtype=torch.bfloat16, device="cuda") for c in (K, N))
    assert sg.grouped_forward(X, Wg, off).shape == (0, N)
    assert sg.grouped_backward_input(dY, Wg, off).shape == (0, K)
    assert not sg.grouped_backward_weight(dY, X, Wg, off).any()
    assert not sg.grouped_bias_grad(dY, off).any()


@pytest.mark.parametrize("T,raw,clamped", [
    (20, [0, 9, 5, 20], [0, 9, 9, 20]), (20, [-4, 3, 8, 99], [0, 3, 8, 20]), (20, [25, 30, 40, 50], [20, 20, 20, 20]),
    (6, [0, 4, 2, 6], [0, 4, 4, 6]), (6, [-1, 2, 3, 2 ** 31 - 1], [0, 2, 3, 6]), (6, [9, 9, -9, 9], [6, 6, 6, 6])])
def test_bad_offsets_are_clamped_and_reported(T, raw, clamped):
    rng = np.random.default_rng(17)
    N, K = 64, 64
    X, _ = normal(rng, (T, K))
    dY, _ = normal(rng, (T, N))
    Wg = sg.GroupedWeight(normal(rng, (3, N, K))[0])
    bad, good = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (raw, clamped))
    for fn in (lambda o: sg.grouped_forward(X, Wg, o), lambda o: sg.grouped_backward_input(dY, Wg, o),
               lambda o: sg.grouped_backward_weight(dY, X, Wg, o)):
        want = fn(good)
        assert sg.grouped_status(Wg) == 0
        assert torch.equal(fn(bad), want)
        assert sg.grouped_status(Wg) == 1   # BSL_ERR_INVALID_ARG, read and cleared
        assert sg.grouped_status(Wg) == 0
    assert torch.equal(sg.grouped_bias_grad(dY, bad), sg.grouped_bias_grad(dY, good))


@pytest.mark.parametrize("rows", [[3, 0, 2], [200, 0, 313]])
def test_repeatable_and_replayed_with_new_offsets(rows):
    """A captured run of the four calls reads the offsets and inputs of the replay, on a stream of its
    own; two such graphs run at once."""
    rng = np.random.default_rng(18)
    N, K = 136, 264
    T = sum(rows)
    Wg = sg.GroupedWeight(normal(rng, (3, N, K))[0])

    def calls(X, dY, off):
        return (sg.grouped_forward(X, Wg, off), sg.grouped_backward_input(dY, Wg, off),
                sg.grouped_backward_weight(dY, X, Wg, off), sg.grouped_bias_grad(dY, off))

    sets = []
    for _ in range(2):
        X, dY = normal(rng, (T, K))[0], normal(rng, (T, N))[0]
        off = offsets_of(rows)[0]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            calls(X, dY, off)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = calls(X, dY, off)
        sets.append((X, dY, off, s, g, outs))
    for new in (rows, rows[::-1], [T, 0, 0], [0, 0, T]):
        for X, dY, off, *_ in sets:
            off.copy_(offsets_of(new)[0])
            X.copy_(normal(rng, (T, K))[0])
            dY.copy_(normal(rng, (T, N))[0])
        torch.cuda.synchronize()
        for *_, s, g, _ in sets:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for X, dY, off, _, _, outs in sets:
            for a, b in zip(outs, calls(X, dY, off)):
                assert torch.equal(a, b)
    assert sg.grouped_status(Wg) == 0


@pytest.mark.parametrize("rows,N,K", [([900, 2100, 0, 40], 4104, 1032), ([4000, 1], 1032, 3000),
                                      ([257] * 12, 2056, 640)])
def test_many_tiles(rows, N, K):
    """Every CTA walks several tiles and its rings wrap many times; a second run has the same bits."""
    first = run_all(rows, N, K, 21)
    for got, ref, S, depth, what in first:
        check(got, ref, S, depth, what)
    for (a, *_), (b, *_) in zip(first, run_all(rows, N, K, 21)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Row starts whose element index passes 2^31."""
    K, N, T = 8192, 16, 270000
    assert T * K > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(3)
    X = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    W = torch.empty(2, N, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dY = torch.empty(T, N, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    Wg = sg.GroupedWeight(W)
    off = torch.tensor([0, T - 37, T], dtype=torch.int32, device="cuda")
    Y = sg.grouped_forward(X, Wg, off)
    dX = sg.grouped_backward_input(dY, Wg, off)
    dW = sg.grouped_backward_weight(dY, X, Wg, off)
    f64 = lambda t: t.double().cpu().numpy()
    tail = slice(T - 60, T)
    o = [0, 23, 60]
    check(Y[tail], *experts.grouped_forward(f64(X[tail]), f64(W), o), K, "Y")
    check(dX[tail], *experts.grouped_backward_input(f64(dY[tail]), f64(W), o), N, "dX")
    last = slice(T - 37, T)
    check(dW[1:], *experts.grouped_backward_weight(f64(dY[last]), f64(X[last]), [0, 37]), 37, "dW")


def test_autograd_and_module():
    """Leading dimensions, padding rows, gradients of the input, weight and bias; the gradients agree
    with differences of the forward (exact on small integers)."""
    rng = np.random.default_rng(19)
    rows, N, K = [7, 0, 12, 4], 72, 40
    off, o = offsets_of(rows)
    T = 24                                        # one padding row
    layer = sg.GroupedLinear(integers(rng, (4, N, K))[0], integers(rng, (4, N))[0])
    X, Xf = integers(rng, (2, T // 2, K))
    dY, dYf = integers(rng, (2, T // 2, N))
    X.requires_grad_(True)
    Y = layer(X, off)
    assert Y.shape == (2, T // 2, N) and not Y.reshape(T, N)[23].any()
    Y.backward(dY)
    Wf, bf = (p.detach().double().cpu().numpy() for p in (layer.weight, layer.bias))
    Xf, dYf = Xf.reshape(T, K), dYf.reshape(T, N)
    f = lambda X, W, b: (experts.grouped_forward(X, W, o, b)[0] * dYf).sum()
    for grad, ref, which in ((X.grad.reshape(T, K), experts.grouped_backward_input(dYf, Wf, o)[0], 0),
                             (layer.weight.grad, experts.grouped_backward_weight(dYf, Xf, o)[0], 1),
                             (layer.bias.grad, experts.grouped_bias_grad(dYf, o)[0], 2)):
        got = grad.double().cpu().numpy()
        check(grad, ref, np.zeros_like(ref), 1, "gradient")
        args = [Xf, Wf, bf]
        h = rng.integers(-2, 3, args[which].shape).astype(float)
        base = f(*args)
        args[which] = args[which] + h
        # bf16 keeps 8 bits of each gradient entry: half a step each
        assert abs((f(*args) - base) - (got * h).sum()) <= 2.0 ** -8 * np.abs(ref * h).sum()
    # an in-place update is what the next call uses; a replaced storage too
    with torch.no_grad():
        layer.weight.mul_(2.0)
        Y2 = layer(X, off)
        layer.weight.data = layer.weight.data.clone()
        Y3 = layer(X, off)
    check(Y2.reshape(T, N)[:23], experts.grouped_forward(Xf[:23], 2 * Wf, o, bf)[0], np.zeros((23, N)), 1, "Y2")
    assert torch.equal(Y2, Y3)


def test_captured_training_step():
    """Forward and backward in one graph: a replay gives the gradients of the inputs it finds."""
    rng = np.random.default_rng(24)
    layer = sg.GroupedLinear(normal(rng, (3, 72, 40))[0], normal(rng, (3, 72))[0])
    X = normal(rng, (200, 40))[0].requires_grad_(True)
    dY = normal(rng, (200, 72))[0]
    off = offsets_of([120, 0, 80])[0]
    params = (X, layer.weight, layer.bias)

    def step():
        layer(X, off).backward(dY)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    for p in params:
        p.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rows in ([120, 0, 80], [0, 37, 163]):
        with torch.no_grad():
            X.copy_(normal(rng, (200, 40))[0])
            dY.copy_(normal(rng, (200, 72))[0])
            off.copy_(offsets_of(rows)[0])
            layer.weight.mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        got = [p.grad.clone() for p in params]
        Wg = layer.packed
        assert torch.equal(got[0], sg.grouped_backward_input(dY, Wg, off))
        assert torch.equal(got[1], sg.grouped_backward_weight(dY, X.detach(), Wg, off))
        assert torch.equal(got[2], sg.grouped_bias_grad(dY, off))


def test_module_copies():
    """Deep copies and pickles of the module work on storage of their own."""
    import copy
    import io
    rng = np.random.default_rng(22)
    layer = sg.GroupedLinear(normal(rng, (2, 16, 24))[0], normal(rng, (2, 16))[0])
    X, _ = normal(rng, (5, 24))
    off = offsets_of([2, 3])[0]
    with torch.no_grad():
        want = layer(X, off)
        buf = io.BytesIO()
        torch.save(layer, buf)
        buf.seek(0)
        for other in (copy.deepcopy(layer), torch.load(buf, weights_only=False)):
            assert torch.equal(other(X, off), want)
            layer.weight.add_(1.0)
            assert torch.equal(other(X, off), want) and not torch.equal(layer(X, off), want)
            layer.weight.copy_(other.weight)


def test_streams_and_strided_gradients():
    """Calls on a stream of their own, and an upstream gradient that is a broadcast."""
    rng = np.random.default_rng(23)
    layer = sg.GroupedLinear(normal(rng, (3, 72, 40))[0], normal(rng, (3, 72))[0])
    X = normal(rng, (50, 40))[0].requires_grad_(True)
    off, o = offsets_of([20, 0, 30])
    layer(X, off).float().sum().backward()
    want = [X.grad.clone(), layer.weight.grad.clone(), layer.bias.grad.clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for p in (X, layer.weight, layer.bias):
        p.grad = None
    with torch.cuda.stream(s):
        layer(X, off).float().sum().backward()
    torch.cuda.current_stream().wait_stream(s)
    for p, w in zip((X, layer.weight, layer.bias), want):
        assert torch.equal(p.grad, w)
    ones = np.ones((50, 72))
    check(want[2], *experts.grouped_bias_grad(ones, o), 16 * 30, "db")
    check(want[0], *experts.grouped_backward_input(ones, layer.weight.detach().double().cpu().numpy(), o), 72, "dX")


def test_refusals():
    W = torch.zeros(2, 16, 24, dtype=torch.bfloat16, device="cuda")
    Wg = sg.GroupedWeight(W)
    X = torch.zeros(5, 24, dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros(5, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (W[0], W.float(), W.cpu()):
        with pytest.raises(TypeError):
            sg.GroupedWeight(bad)
    for bad in (W.transpose(1, 2), W[:, :12], torch.zeros(2, 12, 24, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(1025, 8, 8, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError):
            sg.GroupedWeight(bad)
    for exc, args, kw in (
            (TypeError, (X.float(), Wg, off), {}), (TypeError, (X[0], Wg, off), {}),
            (TypeError, (X, Wg, off.long()), {}), (TypeError, (X, Wg, off.cpu()), {}),
            (ValueError, (X[:, :16], Wg, off), {}), (ValueError, (X, Wg, off[:2]), {}),
            (ValueError, (torch.zeros(24, 5, dtype=torch.bfloat16, device="cuda").t(), Wg, off), {}),
            (ValueError, (X, Wg, off), dict(bias=W[0])), (TypeError, (X, Wg, off), dict(bias=W[:, :, 0].float())),
            (ValueError, (X, Wg, off), dict(out=X)), (TypeError, (X, Wg, off), dict(out=dY.float()))):
        with pytest.raises(exc):
            sg.grouped_forward(*args, **kw)
    with pytest.raises(ValueError):
        sg.grouped_backward_input(X, Wg, off)
    with pytest.raises(ValueError):
        sg.grouped_backward_weight(dY, X[:4], Wg, off)
    with pytest.raises(sg.BslError):
        sg.grouped_bias_grad(dY, off[:1])
    with pytest.raises(ValueError):
        sg.GroupedLinear(W, bias=torch.zeros(2, 24))
    with pytest.raises(ValueError):
        sg.GroupedLinearFunction.apply(X, W.clone(), off, Wg)


def test_out_that_overlaps_an_input_is_refused():
    buf = torch.zeros(64 * 32, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(2, 16, 16, dtype=torch.bfloat16, device="cuda")
    Wg = sg.GroupedWeight(W)
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    X, Y = buf[:128].view(8, 16), buf[64:192].view(8, 16)
    for call in (lambda: sg.grouped_forward(X, Wg, off, out=X), lambda: sg.grouped_forward(X, Wg, off, out=Y),
                 lambda: sg.grouped_forward(X, Wg, off, out=W.view(-1)[:128].view(8, 16)),
                 lambda: sg.grouped_backward_input(X, Wg, off, out=Y),
                 lambda: sg.grouped_backward_weight(buf[1000:1128].view(8, 16), X, Wg, off, out=buf[64:576].view(2, 16, 16)),
                 lambda: sg.grouped_backward_weight(X, buf[1000:1128].view(8, 16), Wg, off, out=buf[64:576].view(2, 16, 16)),
                 lambda: sg.grouped_bias_grad(X, off, out=buf[120:152].view(2, 16))):
        with pytest.raises(ValueError, match="overlap"):
            call()
    sg.grouped_forward(X, Wg, off, out=buf[128:256].view(8, 16))      # neighbours are fine
    assert sg.grouped_status(Wg) == 0


def test_weight_that_changed_its_layout_or_meets_a_capture():
    """A transposed view of the weight's storage is refused; so is a handle made inside a capture."""
    rng = np.random.default_rng(31)
    layer = sg.GroupedLinear(normal(rng, (2, 16, 16))[0])
    X = normal(rng, (8, 16))[0]
    off = offsets_of([3, 5])[0]
    flat = layer.weight.detach()
    with torch.no_grad():
        want = layer(X, off)
        layer.weight.data = flat.transpose(1, 2)
        with pytest.raises(ValueError):
            layer(X, off)
        with pytest.raises(ValueError):
            sg.GroupedLinearFunction.apply(X, layer.weight, off, sg.GroupedWeight(flat))
        layer.weight.data = flat
        assert torch.equal(layer(X, off), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            with pytest.raises(RuntimeError):
                sg.GroupedWeight(flat)
            Y = sg.grouped_forward(X, layer.packed, off)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)
