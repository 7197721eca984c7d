"""GPU parity of the 8-bit layer (e4m3, a scale for each block of 128): conversions bit for bit, products in both
directions against the fp64 oracle, modules.

Products of two e4m3 numbers are exact in fp32, so the bound is that of tests/_experts.py: a block's sum in the tensor
core's additions, one rounding each for the product of the scales, for the scaled sum and for the sum over the blocks
(at most ceil(depth / 128) + 2 of 2^-24, inside the eight additions of 2^-22 and the sixteen-fold count there), and
the rounding to bf16."""
import copy
import io

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


E4M3 = np.array([(-1.0) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if not c & 0x78 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10))
                 for c in range(256)])
E4M3[[0x7F, 0xFF]] = np.nan


def host(q):
    """Code values and scales of an Fp8Tensor."""
    return E4M3[q.codes.view(torch.uint8).cpu().numpy()], q.scales.cpu().numpy()


def assert_quantised(bits, block_rows):
    q = sg.quantize_fp8(to_dev(bits), block_rows=block_rows)
    with np.errstate(invalid="ignore"):
        f = synth.bits_to_f32(bits).astype(np.float64)
    codes, scales = experts.fp8_quantize(f, block_rows)
    got_c, got_s = host(q)
    assert np.array_equal(got_s, scales, equal_nan=True)
    assert np.array_equal(got_c, codes)
    assert np.array_equal(np.signbit(got_c[codes != 0]), np.signbit(codes[codes != 0]))
    v = sg.dequantize_fp8(q).double().cpu().numpy()
    want = experts.fp8_values(codes, scales)
    assert np.array_equal(np.isnan(v), np.isnan(want))
    # one rounding of the product to fp32 and one to bf16
    some = ~np.isnan(want)
    assert (np.abs(v - want)[some] <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)[some]).all()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 144), (37, 128), (130, 272), (300, 1008)])
def test_conversion_bit_exact(rows, K, block_rows):
    rng = np.random.default_rng(rows)
    assert_quantised(synth.bf16_bits((rng.standard_normal((rows, K)) *
                                      np.exp(4 * rng.standard_normal((rows, 1)))).astype(np.float32)), block_rows)


def test_conversion_of_every_bf16_value():
    """Each bf16 number (subnormals, infinities, NaN) beside neighbours of its size, and shuffled; finite ones
    under a block maximum some exponents above."""
    every = np.arange(65536, dtype=np.uint16)
    for block_rows in (1, 128):
        assert_quantised(every.reshape(-1, 128), block_rows)
        assert_quantised(np.random.default_rng(5).permutation(every).reshape(-1, 64), block_rows)
    mag = every[(every & 0x7F80) < 0x7F00]
    blocks = np.resize(mag, (len(mag) + 126) // 127 * 127).reshape(-1, 127)
    top = (blocks & 0x7FFF).max(axis=1).astype(np.int64)
    for up in (0, 3, 8, 12, 17):
        peak = np.minimum(top + 0x80 * up, 0x7F7F)
        assert_quantised(np.ascontiguousarray(np.concatenate([blocks, peak[:, None]], axis=1).astype(np.uint16)), 1)


def test_conversion_of_experts_weights():
    """A stack of planes whose rows end inside a tile: tiles do not reach into the next plane."""
    rng = np.random.default_rng(3)
    bits = synth.bf16_bits((rng.standard_normal((3, 200, 144)) * np.array([1.0, 50.0, 0.02])[:, None, None]).astype(np.float32))
    q = sg.quantize_fp8(to_dev(bits), block_rows=128)
    assert q.shape == (3, 200, 144) and tuple(q.scales.shape) == (3, 2, 2)
    got_c, got_s = host(q)
    for e in range(3):
        codes, scales = experts.fp8_quantize(synth.bits_to_f32(bits[e]).astype(np.float64), 128)
        assert np.array_equal(got_s[e], scales) and np.array_equal(got_c[e], codes)
    by_row = sg.quantize_fp8(to_dev(bits))
    assert tuple(by_row.scales.shape) == (3, 200, 2)


def test_dequantise_every_code():
    codes = torch.arange(256, dtype=torch.uint8).reshape(2, 128).cuda()
    for s in (1.0, 0.3, 2.0 ** -130, 3e38, float("nan"), float("inf")):
        scales = torch.full((2, 1), s, dtype=torch.float32, device="cuda")
        got = sg.dequantize_fp8(sg.Fp8Tensor(codes, scales)).cpu().float().numpy()
        want = torch.from_numpy((E4M3.astype(np.float32) * np.float32(s)).reshape(2, 128)).to(torch.bfloat16).float().numpy()
        assert np.array_equal(got, want, equal_nan=True), s


def weights(rng, *shape):
    """Normal weights in 8 bits, their code values and scales."""
    W, _ = normal(rng, shape, shape[-1] ** -0.5)
    q = sg.quantize_fp8(W, block_rows=128)
    return q, host(q)


def rows_of(rng, T, K, std=1.0):
    X, _ = normal(rng, (T, K), std)
    q = sg.quantize_fp8(X)
    return X, q, host(q)


def reference(rows, weight, offsets=None, transposed=False, bias=None):
    """Product and S of quantised rows and weights (one expert without offsets)."""
    (c, s), (wc, ws) = rows, weight
    if offsets is None:
        y, S = experts.fp8_product(c, s, wc, ws, transposed)
        return (y, S) if bias is None else (y + bias, S + np.abs(bias))
    Y = np.zeros((c.shape[0], wc.shape[2] if transposed else wc.shape[1]))
    S = np.zeros_like(Y)
    for e in range(wc.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        Y[r], S[r] = experts.fp8_product(c[r], s[r], wc[e], ws[e], transposed)
        if bias is not None:
            Y[r] += bias[e]
            S[r] += np.abs(bias[e])
    return Y, S


@pytest.mark.parametrize("M,K,N", [(1, 16, 8), (1, 4096, 1032), (2, 144, 24), (8, 1008, 264), (9, 272, 136), (17, 512, 128),
                                   (31, 128, 256), (33, 144, 520), (65, 256, 264), (100, 640, 712), (257, 1008, 720),
                                   (300, 2064, 376), (513, 128, 1024)])
def test_forward(M, K, N):
    rng = np.random.default_rng(M * 7 + K)
    X, q, xr = rows_of(rng, M, K)
    Wq, wr = weights(rng, N, K)
    bias, bf = normal(rng, (N,))
    ref = reference(xr, wr, bias=bf)
    Y = sg.forward_fp8(X, Wq, bias=bias)
    check(Y, *ref, K, "bf16 rows")
    assert torch.equal(Y, sg.forward_fp8(q, Wq, bias=bias))       # rows quantised before
    out = torch.full_like(Y, float("nan"))
    assert sg.forward_fp8(X, Wq, bias=bias, out=out) is out and torch.equal(out, Y)
    check(sg.forward_fp8(X, Wq), *reference(xr, wr), K, "no bias")
    assert sg.fp8_status(Wq) == 0


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 1040, 512), (3, 144, 48), (16, 272, 1008), (33, 128, 144), (130, 720, 400),
                                   (257, 2064, 272), (300, 256, 1024)])
def test_input_gradient(M, N, K):
    rng = np.random.default_rng(M * 5 + N)
    dY, q, gr = rows_of(rng, M, N, 0.01)
    Wq, wr = weights(rng, N, K)
    dX = sg.backward_input_fp8(dY, Wq)
    check(dX, *reference(gr, wr, transposed=True), N, "dX")
    assert torch.equal(dX, sg.backward_input_fp8(q, Wq))


ROWS = [[1], [0, 1, 0], [3, 0, 2, 1], [9, 0, 5], [16, 17, 0, 31], [40, 1, 90], [0, 0, 129], [255, 1, 256, 257], [300, 0, 33, 7, 140]]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("K,N", [(272, 400), (1008, 144)])
def test_experts(rows, K, N):
    """Both directions, rows of no expert at both ends (NaN there, and left alone in `out`)."""
    rng = np.random.default_rng(sum(rows) + K)
    front, back = 3, 5
    T = front + sum(rows) + back
    off, o = offsets_of(rows, front)
    Wq, wr = weights(rng, len(rows), N, K)
    bias, bf = normal(rng, (len(rows), N))
    rest = np.r_[0:front, T - back:T]
    for depth, cols, transposed in ((K, N, False), (N, K, True)):
        A, _ = normal(rng, (T, depth))
        A[rest] = float("nan")
        q = sg.quantize_fp8(A)
        c, s = host(q)
        c[rest], s[rest] = 0, 0
        ref = reference((c, s), wr, o, transposed, None if transposed else bf)
        call = (lambda a, **kw: sg.grouped_backward_input_fp8(a, Wq, off, **kw)) if transposed else \
            (lambda a, **kw: sg.grouped_forward_fp8(a, Wq, off, bias=bias, **kw))
        Y = call(A)
        check(Y, *ref, depth, f"transposed {transposed}")
        assert not Y[rest].any()
        assert torch.equal(Y, call(q))
        out = torch.full((T, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        call(A, out=out)
        assert (out[rest] == 7).all() and torch.equal(out[front:T - back], Y[front:T - back])
    assert sg.fp8_status(Wq) == 0


@pytest.mark.parametrize("T", [2, 40, 300])
def test_a_rows_nan_stays_in_its_row(T):
    """An infinity in a block of a row, NaN scales and NaN codes of the weight reach their own results only."""
    rng = np.random.default_rng(T)
    K, N = 400, 272
    X, _ = normal(rng, (T, K))
    Wq, wr = weights(rng, N, K)
    clean = sg.forward_fp8(X, Wq)
    X[T // 2, 130] = float("inf")
    Y = sg.forward_fp8(X, Wq)
    assert torch.isnan(Y[T // 2]).all()
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(Y[keep], clean[keep])
    codes = Wq.codes.clone()
    codes.view(torch.uint8)[5, 17] = 0x7F
    codes.view(torch.uint8)[6, 399] = 0xFF
    Yn = sg.forward_fp8(X, sg.Fp8Tensor(codes, Wq.scales))
    assert torch.isnan(Yn[:, 5:7]).all()
    keep_n = torch.ones(N, dtype=torch.bool, device="cuda")
    keep_n[5:7] = False
    assert torch.equal(Yn[keep][:, keep_n], clean[keep][:, keep_n])
    scales = Wq.scales.clone()
    scales[1, 2] = float("nan")   # features 128 .. 255
    Ys = sg.forward_fp8(X, sg.Fp8Tensor(Wq.codes, scales))
    assert torch.isnan(Ys[:, 128:256]).all() and torch.equal(Ys[keep][:, :128], clean[keep][:, :128])
    assert torch.equal(Ys[keep][:, 256:], clean[keep][:, 256:])


@pytest.mark.parametrize("offsets,T", [([0, 50, 30, 60], 60), ([-5, 20, 90, 70], 60), ([10, 10, 700, 5], 60), ([0, 2, 9, 3], 4)])
def test_bad_offsets_are_clamped_and_reported(offsets, T):
    rng = np.random.default_rng(1)
    Wq, wr = weights(rng, 3, 144, 272)
    for depth, transposed in ((272, False), (144, True)):
        X, q, xr = rows_of(rng, T, depth)
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        safe = np.maximum.accumulate(np.clip(offsets, 0, T))
        call = sg.grouped_backward_input_fp8 if transposed else sg.grouped_forward_fp8
        check(call(X, Wq, off), *reference(xr, wr, safe, transposed), depth, "clamped")
        assert sg.fp8_status(Wq) == 1 and sg.fp8_status(Wq) == 0


def test_no_rows():
    rng = np.random.default_rng(2)
    Wq, _ = weights(rng, 2, 144, 272)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    X = torch.empty(0, 272, dtype=torch.bfloat16, device="cuda")
    assert sg.grouped_forward_fp8(X, Wq, off).shape == (0, 144)
    assert sg.grouped_forward_fp8(sg.quantize_fp8(X), Wq, off).shape == (0, 144)
    assert sg.dequantize_fp8(sg.quantize_fp8(X)).shape == (0, 272)
    Z = torch.ones(70, 272, dtype=torch.bfloat16, device="cuda")
    assert not sg.grouped_forward_fp8(Z, Wq, off).any() and not sg.grouped_forward_fp8(Z[:4], Wq, off).any()


def test_more_tiles_than_ctas_and_long_sums():
    """Several tiles a CTA, an odd number of blocks a tile: the accumulators' turns go on over tiles."""
    rng = np.random.default_rng(8)
    X, q, xr = rows_of(rng, 1100, 4112)
    Wq, wr = weights(rng, 4360, 4112)
    Y = sg.forward_fp8(q, Wq)
    pick = np.r_[0:5, 250:262, 1095:1100]
    check(Y[pick], *reference((xr[0][pick], xr[1][pick]), wr), 4112, "rows")
    assert all(torch.equal(Y, sg.forward_fp8(q, Wq)) for _ in range(3))
    g, gq, gr = rows_of(rng, 700, 4368, 0.01)
    W2, w2 = weights(rng, 4368, 2064)
    check(sg.backward_input_fp8(gq, W2)[pick[:12]], *reference((gr[0][pick[:12]], gr[1][pick[:12]]), w2, transposed=True), 4368,
          "dX")


def test_unaligned_outputs_and_streams():
    """An output that begins 16 bytes off a 32-byte boundary; another stream than the default one."""
    rng = np.random.default_rng(4)
    X, q, xr = rows_of(rng, 70, 256)
    Wq, wr = weights(rng, 272, 256)
    buf = torch.zeros(70 * 272 + 16, dtype=torch.bfloat16, device="cuda")
    out = buf[8:8 + 70 * 272].view(70, 272)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sg.forward_fp8(X, Wq, out=out)
    s.synchronize()
    check(out, *reference(xr, wr), 256, "off by 16")
    assert not buf[:8].any() and not buf[-8:].any()


def test_modules():
    rng = np.random.default_rng(9)
    W, _ = normal(rng, (272, 144))
    bias, _ = normal(rng, (272,))
    layer = sg.Fp8Linear.from_dense(W, bias)
    x, _ = normal(rng, (3, 11, 144))
    x.requires_grad_(True)
    y = layer(x)
    Wq = sg.quantize_fp8(W, block_rows=128)
    flat = x.detach().reshape(-1, 144)
    assert torch.equal(y.detach(), sg.forward_fp8(flat, Wq, bias=bias).view(3, 11, 272))
    g, _ = normal(rng, (3, 11, 272))
    y.backward(g)
    assert torch.equal(x.grad, sg.backward_input_fp8(g.view(-1, 272), Wq).view(3, 11, 144))
    # state, copies, casts and moves carry the weight
    assert set(layer.state_dict()) == {"codes", "scales", "bias"}
    other = sg.Fp8Linear.from_dense(torch.zeros_like(W), torch.zeros_like(bias))
    other.load_state_dict(layer.state_dict())
    buf = io.BytesIO()
    torch.save(layer, buf)
    buf.seek(0)
    for m in (other, copy.deepcopy(layer), torch.load(buf, weights_only=False), layer.float(), layer.cpu().cuda()):
        assert torch.equal(m(x.detach()), y.detach())


def test_grouped_module_gradient():
    rng = np.random.default_rng(10)
    rows = [5, 0, 70, 33]
    off, o = offsets_of(rows, 2)
    T = sum(rows) + 4
    W, _ = normal(rng, (4, 144, 272))
    layer = sg.GroupedFp8Linear.from_dense(W)
    x, _ = normal(rng, (T, 272))
    x.requires_grad_(True)
    y = layer(x.float(), off)
    g, _ = normal(rng, (T, 144))
    y.backward(g)
    gq = host(sg.quantize_fp8(g))
    check(x.grad, *reference(gq, host(layer.weight8), o, True), 144, "dX")
    odd = sg.GroupedFp8Linear.from_dense(W[:, :136].contiguous())
    assert odd(x.detach(), off).shape == (T, 136)
    with pytest.raises(ValueError, match="multiples of 16"):
        odd(x, off)


def test_capture_and_replay():
    """Two graphs over one weight, each with its own rows and workspace, replayed in turn."""
    rng = np.random.default_rng(12)
    Wq, wr = weights(rng, 3, 144, 272)
    Wq.status
    off, o = offsets_of([20, 0, 60])
    graphs = []
    for i in range(2):
        X, _ = normal(rng, (80, 272))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y = sg.grouped_forward_fp8(X, Wq, off)
            dX = sg.grouped_backward_input_fp8(Y, Wq, off)
        graphs.append((g, X, Y, dX))
    for rep in range(3):
        for g, X, Y, dX in graphs:
            X.copy_(normal(rng, (80, 272))[0])
            g.replay()
        torch.cuda.synchronize()
        for g, X, Y, dX in graphs:
            assert torch.equal(Y, sg.grouped_forward_fp8(X, Wq, off))
            assert torch.equal(dX, sg.grouped_backward_input_fp8(Y, Wq, off))


def test_refusals():
    rng = np.random.default_rng(13)
    Wq, _ = weights(rng, 144, 272)
    Wg, _ = weights(rng, 2, 136, 272)
    X, _ = normal(rng, (4, 272))
    off, _ = offsets_of([2, 2])
    for bad, what in ((lambda: sg.forward_fp8(X[:, :256], Wq), ValueError), (lambda: sg.forward_fp8(X.float(), Wq), TypeError),
                      (lambda: sg.forward_fp8(X, Wg), ValueError), (lambda: sg.grouped_forward_fp8(X, Wq, off), ValueError),
                      (lambda: sg.grouped_forward_fp8(X, Wg, off.long()), TypeError),
                      (lambda: sg.grouped_forward_fp8(X, Wg, off[:2]), ValueError),
                      (lambda: sg.forward_fp8(X.t().contiguous().t(), Wq), ValueError),
                      (lambda: sg.forward_fp8(X, Wq, out=X), ValueError), (lambda: sg.forward_fp8(X, sg.quantize_fp8(X)), ValueError),
                      (lambda: sg.forward_fp8(sg.quantize_fp8(X.repeat(50, 1), block_rows=128), Wq), ValueError),
                      (lambda: sg.grouped_backward_input_fp8(torch.zeros(4, 136, dtype=torch.bfloat16, device="cuda"), Wg, off), ValueError),
                      (lambda: sg.quantize_fp8(X, block_rows=64), ValueError), (lambda: sg.quantize_fp8(X[:, :8].contiguous()), ValueError),
                      (lambda: sg.Fp8Tensor(Wq.codes, Wq.scales[:1]), ValueError),
                      (lambda: sg.Fp8Tensor(Wq.codes, Wq.scales.double()), TypeError),
                      (lambda: sg.forward_fp8(X, Wq, bias=torch.zeros(8, dtype=torch.bfloat16, device="cuda")), ValueError)):
        with pytest.raises(what):
            bad()
    with pytest.raises(sg.BslError):   # 8 bytes off a 16-byte boundary
        flat = torch.zeros(4 * 272 + 4, dtype=torch.bfloat16, device="cuda")[4:]
        sg.forward_fp8(flat.view(4, 272), Wq)
