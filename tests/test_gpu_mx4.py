"""GPU parity of the microscaled 4-bit layer: conversions bit for bit, products
against the fp64 oracle, modules, and experts trained in bf16 and served in 4 bits."""
import numpy as np
import pytest
import torch

import synth
from oracle import experts
from tests._experts import check, normal, offsets_of
from tests._gpu import to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def host(q):
    return q.codes.cpu().numpy(), q.scales.cpu().numpy()


def assert_quantised(bits):
    X = to_dev(bits)
    q = sg.quantize_mx4(X)
    with np.errstate(invalid="ignore"):
        f = synth.bits_to_f32(bits).astype(np.float64)
    codes, scales = experts.mx4_quantize(f)
    got_c, got_s = host(q)
    assert np.array_equal(got_s, scales)
    assert np.array_equal(got_c, codes)
    v = sg.dequantize_mx4(q)
    want = experts.mx4_values(codes, scales)
    nan = np.isnan(want)
    back = v.double().cpu().numpy()
    assert np.array_equal(np.isnan(back), nan)
    assert np.array_equal(back[~nan], want[~nan])
    assert np.array_equal(np.signbit(back[~nan]), np.signbit(want[~nan]))


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (33, 64), (257, 160)])
def test_conversion_bit_exact(rows, K):
    rng = np.random.default_rng(rows)
    assert_quantised(synth.bf16_bits((rng.standard_normal((rows, K)) *
                                      np.exp(4 * rng.standard_normal((rows, 1)))).astype(np.float32)))


def test_conversion_of_every_bf16_value():
    """Each bf16 number (subnormals, infinities, NaN) beside neighbours of its size, and shuffled."""
    every = np.arange(65536, dtype=np.uint16)
    assert_quantised(every.reshape(-1, 64))
    assert_quantised(np.random.default_rng(5).permutation(every).reshape(-1, 128))
    # finite ones only, each under a block maximum one to four exponents above
    mag = every[(every & 0x7F80) < 0x7F80]
    blocks = np.resize(mag, (len(mag) + 29) // 30 * 30).reshape(-1, 30)
    top = blocks.max(axis=1, initial=0, where=blocks < 0x8000)
    up = np.minimum((top.astype(np.int64) & 0x7F80) + 0x80 * np.random.default_rng(6).integers(1, 5, len(top)), 0x7F00)
    rows = np.concatenate([blocks, up[:, None], -up[:, None] & 0x7FFF | 0x8000], axis=1).astype(np.uint16)
    assert_quantised(np.ascontiguousarray(rows))


def test_dequantise_every_scale():
    codes = np.tile(np.arange(16, dtype=np.uint8) | np.arange(15, -1, -1, dtype=np.uint8) << 4, (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    q = sg.Mx4Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    want = torch.from_numpy(experts.mx4_values(codes, scales)).float().to(torch.bfloat16)
    got = sg.dequantize_mx4(q).cpu()
    assert torch.equal(torch.nan_to_num(got, nan=0.5), torch.nan_to_num(want, nan=0.5))
    assert torch.equal(torch.isnan(got), torch.isnan(want))


def weights(rng, *shape):
    """Quantised normal weights and their values (the conversion has its own tests)."""
    W, _ = normal(rng, shape, shape[-1] ** -0.5)
    q = sg.quantize_mx4(W)
    return q, experts.mx4_values(*host(q))


def rows_of(rng, T, K):
    x = rng.standard_normal((T, K)) * np.exp(rng.standard_normal((T, 1)))
    return to_dev(synth.bf16_bits(x.astype(np.float32)))


DENSE = [(1, 8, 32, False), (1, 136, 4096, True), (3, 264, 96, True), (16, 520, 288, False), (33, 128, 256, True),
         (129, 256, 512, False), (200, 72, 1056, True), (500, 1032, 160, True), (1000, 392, 768, False)]


@pytest.mark.parametrize("M,N,K,with_bias", DENSE)
def test_dense_parity(M, N, K, with_bias):
    rng = np.random.default_rng(M + N)
    Wq, Wf = weights(rng, N, K)
    X = rows_of(rng, M, K)
    b, bf = normal(rng, (N,)) if with_bias else (None, None)
    Xq = sg.quantize_mx4(X)
    Y = sg.forward_mx4(X, Wq, bias=b)
    assert torch.equal(Y, sg.forward_mx4(Xq, Wq, bias=b))
    assert sg.mx4_status(Wq) == 0
    Xf = experts.mx4_values(*host(Xq))
    ref, S = Xf @ Wf.T, np.abs(Xf) @ np.abs(Wf).T
    if with_bias:
        ref, S = ref + bf, S + np.abs(bf)
    check(Y, ref, S, K, "mx4")


GROUPED = [
    ([1], 8, 32, 0, 0), ([0, 1, 0], 72, 64, 0, 0), ([3, 0, 2], 264, 96, 2, 3), ([1] * 8, 136, 544, 0, 0),
    ([16, 17, 15, 0, 31, 33], 136, 224, 0, 5), ([63, 64, 65, 127, 128, 129], 128, 64, 1, 0),
    ([191, 192, 193, 0, 255, 256, 257], 256, 128, 0, 0), ([300, 5, 0, 700], 520, 992, 0, 37), ([0, 0], 64, 64, 4, 4),
    ([2, 0, 0, 90], 2056, 320, 0, 0),
]


@pytest.mark.parametrize("rows,N,K,first,spare", GROUPED)
def test_grouped_parity(rows, N, K, first, spare):
    rng = np.random.default_rng(N + K)
    E = len(rows)
    off, o = offsets_of(rows, first)
    T = int(o[-1]) + spare
    Wq, Wf = weights(rng, E, N, K)
    X = rows_of(rng, T, K)
    b, bf = normal(rng, (E, N)) if spare else (None, None)
    Y = sg.grouped_forward_mx4(X, Wq, off, bias=b)
    assert sg.mx4_status(Wq) == 0
    Xf = experts.mx4_values(*host(sg.quantize_mx4(X)))
    check(Y, *experts.grouped_forward(Xf, Wf, o, bf), K, "grouped mx4")
    # rows of no expert stay as they are in a given output
    frame = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    sg.grouped_forward_mx4(X, Wq, off, bias=b, out=frame[1:T + 1])
    assert torch.equal(frame[1 + first:1 + int(o[-1])], Y[first:int(o[-1])])
    assert (frame[:1 + first] == 7.0).all() and (frame[1 + int(o[-1]):] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(3000, 4104, 4096), (1500, 9000, 1312), (9000, 1032, 2560), (2000, 5000, 96)])
def test_many_tiles(M, N, K):
    """Every CTA walks several tiles and its rings wrap many times; all rows of a band of features and
    all features of some rows are compared, and a second run has the same bits."""
    rng = np.random.default_rng(M)
    Wq, Wf = weights(rng, N, K)
    X = rows_of(rng, M, K)
    Xq = sg.quantize_mx4(X)
    Y = sg.forward_mx4(Xq, Wq)
    assert torch.equal(Y, sg.forward_mx4(Xq, Wq))
    assert sg.mx4_status(Wq) == 0
    Xf = experts.mx4_values(*host(Xq))
    cols = slice(N - 300, N)
    check(Y[:, cols], Xf @ Wf[cols].T, np.abs(Xf) @ np.abs(Wf[cols]).T, K, "features")
    rows = sorted({0, 223, 224, M // 2, M - 33, M - 1})
    check(Y[rows], Xf[rows] @ Wf.T, np.abs(Xf[rows]) @ np.abs(Wf).T, K, "rows")


@pytest.mark.parametrize("rows,N,K,first,spare", [
    ([8], 1032, 4096, 0, 0), ([1], 11008, 4096, 0, 0), ([0, 3, 0, 0, 1, 0, 2], 520, 2080, 1, 1),
    ([0] * 31 + [2] + [0] * 200 + [1, 0, 3], 72, 160, 0, 2), ([0] * 1000 + [5], 16, 32, 2, 1), ([9], 136, 992, 0, 0),
    ([3, 0, 11], 264, 992, 1, 1), ([16], 1032, 512, 0, 0), ([16], 4104, 2080, 0, 0), ([17], 136, 512, 0, 0)])
def test_few_rows(rows, N, K, first, spare):
    rng = np.random.default_rng(N + K + first)
    off, o = offsets_of(rows, first)
    Wq, Wf = weights(rng, len(rows), N, K)
    X = rows_of(rng, int(o[-1]) + spare, K)
    b, bf = normal(rng, (len(rows), N))
    Xf = experts.mx4_values(*host(sg.quantize_mx4(X)))
    Y = sg.grouped_forward_mx4(X, Wq, off, bias=b)
    check(Y, *experts.grouped_forward(Xf, Wf, o, bf), K, "few rows")
    assert not Y[:first].any() and not Y[int(o[-1]):].any()
    assert sg.mx4_status(Wq) == 0


@pytest.mark.parametrize("M", [3, 12, 40])
def test_every_scale_byte(M):
    """Weight rows and activation rows under every scale byte whose products stay in the fp32 range."""
    rng = np.random.default_rng(M)
    N, K = 256, 64
    codes = lambda r: torch.from_numpy(rng.integers(0, 256, (r, K // 2), dtype=np.uint8)).cuda()
    for xs in (0, 1, 60, 127, 128, 129, 180, 250):
        byte = np.arange(N)
        ok = (byte + xs > 20) & (byte + xs < 360) & (byte < 255)      # 2^-234 .. 2^106
        ws = np.where(ok, byte, 127).astype(np.uint8)
        Wq = sg.Mx4Tensor(codes(N), torch.from_numpy(np.repeat(ws[:, None], 2, axis=1)).cuda())
        Xq = sg.Mx4Tensor(codes(M), torch.full((M, 2), xs, dtype=torch.uint8, device="cuda"))
        Xf, Wf = experts.mx4_values(*host(Xq)), experts.mx4_values(*host(Wq))
        ref, S = Xf @ Wf.T, np.abs(Xf) @ np.abs(Wf).T
        Y = sg.forward_mx4(Xq, Wq)
        unit = ws.astype(int) + xs - 254
        fits = (unit > -110) & (unit < 110)          # far above the subnormal numbers, below the fp32 range
        check(Y[:, fits], ref[:, fits], S[:, fits], K, f"scale {xs}")
        assert (Y[:, unit <= -110].double().abs().cpu().numpy() <= 2.0 ** -100).all()
        # past the fp32 range: not finite (an infinity has the sign of the partial sum that passed it)
        assert not np.isfinite(Y.double().cpu().numpy()[np.abs(ref) > 2.0 ** 129]).any()


def test_many_experts():
    rng = np.random.default_rng(7)
    rows = rng.integers(0, 3, 1024).tolist()
    off, o = offsets_of(rows)
    Wq, Wf = weights(rng, 1024, 16, 32)
    X = rows_of(rng, int(o[-1]), 32)
    Xf = experts.mx4_values(*host(sg.quantize_mx4(X)))
    check(sg.grouped_forward_mx4(X, Wq, off), *experts.grouped_forward(Xf, Wf, o), 32, "many experts")


@pytest.mark.parametrize("M", [5, 15, 300])
def test_nan_blocks_and_extreme_scales(M):
    """A NaN or an infinity in a row makes that row NaN and no other; scale bytes at both ends count."""
    rng = np.random.default_rng(8)
    N, K = 264, 320
    Wq, Wf = weights(rng, N, K)
    X = rows_of(rng, M, K)
    X[1, 5] = float("nan")
    X[3, 310] = float("-inf")
    X[2] *= 2.0 ** -120
    X[4] = 0
    Xq = sg.quantize_mx4(X)
    Xf = experts.mx4_values(*host(Xq))
    Y = sg.forward_mx4(Xq, Wq)
    bad = [1, 3]
    assert torch.isnan(Y[bad].float()).all()
    keep = [r for r in range(M) if r not in bad]
    ref, S = Xf[keep] @ Wf.T, np.abs(Xf[keep]) @ np.abs(Wf).T
    check(Y[keep], ref, S, K, "rows beside NaN rows")
    assert not Y[4].any()
    Wq.scales[7, 2] = 255                     # a NaN block of the weight: that feature only
    Y2 = sg.forward_mx4(Xq, Wq)
    assert torch.isnan(Y2[:, 7].float()).all()
    others = [n for n in range(N) if n != 7]
    assert torch.equal(Y2[keep][:, others], Y[keep][:, others])


@pytest.mark.parametrize("rows", [[4, 0, 3], [150, 0, 250]])
def test_replayed_with_new_inputs(rows):
    rng = np.random.default_rng(9)
    N, K, T = 136, 288, sum(rows)
    Wq, _ = weights(rng, 3, N, K)
    X, off = rows_of(rng, T, K), offsets_of(rows)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sg.grouped_forward_mx4(X, Wq, off)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        Y = sg.grouped_forward_mx4(X, Wq, off)
    for new in (rows, rows[::-1], [0, T, 0]):
        off.copy_(offsets_of(new)[0])
        X.copy_(rows_of(rng, T, K))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, sg.grouped_forward_mx4(X, Wq, off))
    assert sg.mx4_status(Wq) == 0


@pytest.mark.parametrize("T,raw,clamped", [(20, [-1, 9, 5, 77], [0, 9, 9, 20]), (6, [-1, 4, 2, 77], [0, 4, 4, 6])])
def test_bad_offsets_are_clamped_and_reported(T, raw, clamped):
    rng = np.random.default_rng(10)
    Wq, _ = weights(rng, 3, 64, 64)
    X = rows_of(rng, T, 64)
    bad, good = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (raw, clamped))
    want = sg.grouped_forward_mx4(X, Wq, good)
    assert sg.mx4_status(Wq) == 0
    assert torch.equal(sg.grouped_forward_mx4(X, Wq, bad), want)
    assert sg.mx4_status(Wq) == 1
    assert sg.mx4_status(Wq) == 0


def test_no_rows():
    Wq = sg.quantize_mx4(torch.ones(2, 64, 32, dtype=torch.bfloat16, device="cuda"))
    X = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    assert sg.quantize_mx4(X).shape == (0, 32)
    assert sg.dequantize_mx4(sg.quantize_mx4(X)).shape == (0, 32)
    assert sg.grouped_forward_mx4(X, Wq, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 64)
    assert sg.Mx4Linear.from_dense(torch.ones(64, 32, device="cuda"))(X).shape == (0, 64)


def test_trained_experts_served_in_4_bits():
    """An expert MLP: forward and backward in bf16 through the layers, then both products in 4 bits
    from the same weights, each step against the oracle on the step's own inputs."""
    rng = np.random.default_rng(11)
    rows, K, H = [40, 0, 9, 23], 96, 160
    off, o = offsets_of(rows)
    T = int(o[-1])
    up = sg.GroupedLinear(normal(rng, (4, H, K), K ** -0.5)[0], normal(rng, (4, H))[0])
    down = sg.GroupedLinear(normal(rng, (4, K, H), H ** -0.5)[0])
    x = rows_of(rng, T, K).requires_grad_(True)
    h = up(x, off)
    a = torch.relu(h)
    a.retain_grad()
    h.retain_grad()
    y = down(a, off)
    dy = normal(rng, (T, K))[0]
    y.backward(dy)
    f64 = lambda t: t.detach().double().cpu().numpy()
    check(h, *experts.grouped_forward(f64(x), f64(up.weight), o, f64(up.bias)), K, "up")
    check(y, *experts.grouped_forward(f64(a), f64(down.weight), o), H, "down")
    check(a.grad, *experts.grouped_backward_input(f64(dy), f64(down.weight), o), K, "da")
    depth = np.asarray(rows, dtype=float)[:, None, None]
    check(down.weight.grad, *experts.grouped_backward_weight(f64(dy), f64(a), o), depth, "d down")
    check(up.weight.grad, *experts.grouped_backward_weight(f64(h.grad), f64(x), o), depth, "d up")
    check(up.bias.grad, *experts.grouped_bias_grad(f64(h.grad), o), 16 * depth[:, 0], "d up bias")
    check(x.grad, *experts.grouped_backward_input(f64(h.grad), f64(up.weight), o), H, "dx")
    up4 = sg.GroupedMx4Linear.from_dense(up.weight, up.bias)
    down4 = sg.GroupedMx4Linear.from_dense(down.weight)
    h4 = up4(x.reshape(2, T // 2, K), off)
    a4 = torch.relu(h4)
    y4 = down4(a4, off)
    assert y4.shape == (2, T // 2, K)
    for got, inp, layer, bias, depth in ((h4, x, up, f64(up.bias), K), (y4, a4, down, None, H)):
        inp = inp.detach().reshape(T, -1)
        xq = experts.mx4_values(*experts.mx4_quantize(f64(inp)))
        wq = experts.mx4_values(*experts.mx4_quantize(f64(layer.weight).reshape(-1, depth)))
        check(got.reshape(T, -1), *experts.grouped_forward(xq, wq.reshape(4, -1, depth), o, bias), depth, "served")


def test_linear_module_follows_the_dense_layer():
    rng = np.random.default_rng(12)
    W, b = normal(rng, (72, 128), 0.1)[0], normal(rng, (72,))[0]
    mod = sg.Mx4Linear.from_dense(W.float(), b)
    x = rows_of(rng, 30, 128)
    y = mod(x.float().reshape(2, 3, 5, 128))
    assert y.shape == (2, 3, 5, 72)
    assert torch.equal(y.reshape(30, 72), sg.forward_mx4(x, sg.quantize_mx4(W), bias=b))


def test_copies_and_views():
    """codes and scales of a quantised tensor are views of it; copies and pickles stand on their own; a
    weight whose first use would be captured is refused, one that was used is not."""
    import copy
    import io
    rng = np.random.default_rng(13)
    W, X = normal(rng, (72, 96))[0], rows_of(rng, 20, 96)
    q = sg.quantize_mx4(W)
    assert q.codes.shape == (72, 48) and q.scales.shape == (72, 3)
    mod = sg.Mx4Linear(q)
    want = mod(X)
    buf = io.BytesIO()
    torch.save(mod, buf)
    buf.seek(0)
    others = [copy.deepcopy(mod), torch.load(buf, weights_only=False)]
    q.scales.sub_(1)                              # half of every value
    assert torch.equal(mod(X), want / 2)
    assert torch.equal(sg.dequantize_mx4(q), sg.dequantize_mx4(others[0].weight4) / 2)
    for m in others:
        assert torch.equal(m(X), want)
    fresh = sg.quantize_mx4(W)
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before capturing"):
        with torch.cuda.graph(g):
            sg.forward_mx4(X, fresh)
    torch.cuda.synchronize()
    fresh.status
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = sg.forward_mx4(X, fresh)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


def test_refusals():
    codes = torch.zeros(4, 16, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(4, 1, dtype=torch.uint8, device="cuda")
    q = sg.Mx4Tensor(codes, scales)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    for exc, args in ((TypeError, (codes[0], scales[0])), (TypeError, (codes.int(), scales)),
                      (ValueError, (codes[:, :8], scales)), (ValueError, (codes, scales[:3])),
                      (ValueError, (codes.t().contiguous().t(), scales)), (TypeError, (codes, scales.int()))):
        with pytest.raises(exc):
            sg.Mx4Tensor(*args)
    for exc, x in ((ValueError, bf(4, 48)), (TypeError, bf(4, 64).float()), (ValueError, bf(64, 4).t()),
                   (TypeError, bf(64)), (ValueError, bf(4, 0))):
        with pytest.raises(exc):
            sg.quantize_mx4(x)
    with pytest.raises(ValueError):
        sg.quantize_mx4(bf(5, 32), out=q)
    with pytest.raises(ValueError):
        sg.dequantize_mx4(q, out=bf(4, 64))
    with pytest.raises(sg.BslError):
        sg.forward_mx4(bf(2, 32), q)                         # 4 features: not a multiple of 8
    w = sg.quantize_mx4(bf(8, 32))
    w3 = sg.quantize_mx4(bf(2, 8, 32))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: sg.forward_mx4(bf(2, 64), w), lambda: sg.forward_mx4(bf(2, 32), w3),
                 lambda: sg.forward_mx4(sg.quantize_mx4(bf(2, 64)), w), lambda: sg.forward_mx4(w3, w),
                 lambda: sg.forward_mx4(bf(2, 32), w, out=bf(3, 8)),
                 lambda: sg.grouped_forward_mx4(bf(2, 32), w, off),
                 lambda: sg.grouped_forward_mx4(bf(2, 32), w3, off[:2]),
                 lambda: sg.grouped_forward_mx4(bf(2, 32), w3, off, bias=bf(2, 16)),
                 lambda: sg.Mx4Linear.from_dense(bf(8, 32), bf(9))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sg.forward_mx4(bf(2, 32).float(), w), lambda: sg.forward_mx4(bf(2, 32), w, bias=bf(9)),
                 lambda: sg.grouped_forward_mx4(bf(2, 32), w3, off.long())):
        with pytest.raises(TypeError):
            call()


def test_out_that_overlaps_an_input_is_refused():
    X = torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")
    q = sg.quantize_mx4(X)
    w = sg.quantize_mx4(torch.zeros(32, 32, dtype=torch.bfloat16, device="cuda"))
    inside = q._held[:64].view(2, 32)
    for call in (lambda: sg.forward_mx4(X, w, out=X), lambda: sg.dequantize_mx4(sg.Mx4Tensor(q.codes[:2], q.scales[:2]), out=inside),
                 lambda: sg.forward_mx4(sg.Mx4Tensor(q.codes[:2], q.scales[:2]), w, out=inside)):
        with pytest.raises(ValueError, match="overlap"):
            call()


@pytest.mark.parametrize("K", [256, 768, 11008, 128, 640, 1152, 64, 320, 32, 96, 1440, 2848])
@pytest.mark.parametrize("M", [3, 11, 37, 301])
def test_scale_rows_of_every_length(M, K):
    """Rows of scales in units of 16, 8, 4, 2 and 1 bytes: the bytes of the next row, NaN there, reach
    nobody, and the last row's end with the array."""
    rng = np.random.default_rng(M + K)
    N = 264
    Wq, _ = weights(rng, N, K)
    Xq = sg.quantize_mx4(rows_of(rng, M, K))
    Wq.scales[5] = 255
    Xq.scales[1] = 255
    Xf, Wf = experts.mx4_values(*host(Xq)), experts.mx4_values(*host(Wq))
    Y = sg.forward_mx4(Xq, Wq)
    rows, cols = [r for r in range(M) if r != 1], [n for n in range(N) if n != 5]
    assert torch.isnan(Y[1].float()).all() and torch.isnan(Y[:, 5].float()).all()
    Xk, Wk = Xf[rows], Wf[cols]
    check(Y[rows][:, cols], Xk @ Wk.T, np.abs(Xk) @ np.abs(Wk).T, K, "other rows and features")
    assert sg.mx4_status(Wq) == 0
