"""Pins of the expert-layer and 4-bit oracles, and host-side refusals of their
entry points (no GPU: every check precedes the first CUDA call)."""
import ctypes
import math
import re
import os
from fractions import Fraction

import numpy as np
import pytest

from oracle import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_grouped_products_against_integer_loops():
    rng = np.random.default_rng(1)
    offsets, N, K, T = [1, 4, 4, 6], 3, 2, 8
    X, dY = rng.integers(-3, 4, (T, K)), rng.integers(-3, 4, (T, N))
    W, b = rng.integers(-3, 4, (3, N, K)), rng.integers(-3, 4, (3, N))
    Y, _ = experts.grouped_forward(X.astype(float), W.astype(float), offsets, b.astype(float))
    dX, _ = experts.grouped_backward_input(dY.astype(float), W.astype(float), offsets)
    dW, _ = experts.grouped_backward_weight(dY.astype(float), X.astype(float), offsets)
    db, _ = experts.grouped_bias_grad(dY.astype(float), offsets)
    owner = [None, 0, 0, 0, 2, 2, None, None]
    for t, e in enumerate(owner):
        for n in range(N):
            want = 0 if e is None else sum(int(X[t, k]) * int(W[e, n, k]) for k in range(K)) + int(b[e, n])
            assert Y[t, n] == want
        for k in range(K):
            assert dX[t, k] == (0 if e is None else sum(int(dY[t, n]) * int(W[e, n, k]) for n in range(N)))
    for e in range(3):
        rows = [t for t, o in enumerate(owner) if o == e]
        for n in range(N):
            assert db[e, n] == sum(int(dY[t, n]) for t in rows)
            for k in range(K):
                assert dW[e, n, k] == sum(int(dY[t, n]) * int(X[t, k]) for t in rows)


def test_grouped_gradients_against_differences():
    """<dY, Y(X + h) - Y(X)> = <dX, h>, and the same for W and the bias (all exact on integers)."""
    rng = np.random.default_rng(2)
    offsets, N, K, T, E = [0, 3, 3, 7], 4, 5, 9, 3
    draw = lambda *s: rng.integers(-3, 4, s).astype(float)
    X, W, b, dY, hX, hW, hb = (draw(T, K), draw(E, N, K), draw(E, N), draw(T, N), draw(T, K), draw(E, N, K), draw(E, N))
    f = lambda X, W, b: (experts.grouped_forward(X, W, offsets, b)[0] * dY).sum()
    assert f(X + hX, W, b) - f(X, W, b) == (experts.grouped_backward_input(dY, W, offsets)[0] * hX).sum()
    assert f(X, W + hW, b) - f(X, W, b) == (experts.grouped_backward_weight(dY, X, offsets)[0] * hW).sum()
    assert f(X, W, b + hb) - f(X, W, b) == (experts.grouped_bias_grad(dY, offsets)[0] * hb).sum()


def _block(values):
    return [float(v) for v in values] + [0.0] * (32 - len(values))


def test_mx4_rounding_by_hand():
    # scale 1 (largest magnitude in 4 .. 8): every level, every tie, both signs, saturation
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    codes, s = experts.mx4_block(_block([7.5, -7.5, 6, 4, 3, 2, 1.5, 1, .5, 0] + ties + [-t for t in ties]))
    assert s == 127
    assert codes[:10] == [7, 15, 7, 6, 5, 4, 3, 2, 1, 0]
    assert codes[10:17] == [0, 2, 2, 4, 4, 6, 6]
    assert codes[17:24] == [8, 10, 10, 12, 12, 14, 14]


def test_mx4_scales_by_hand():
    assert experts.mx4_block(_block([1.0]))[1] == 125          # 2^0 -> 2^-2
    assert experts.mx4_block(_block([math.nextafter(2.0, 0)]))[1] == 125
    assert experts.mx4_block(_block([2.0]))[1] == 126
    assert experts.mx4_block(_block([]))[1] == 0
    assert experts.mx4_block(_block([2.0 ** -125]))[1] == 0
    assert experts.mx4_block(_block([2.0 ** -124]))[1] == 1
    assert experts.mx4_block(_block([2.0 ** 127]))[1] == 252
    assert experts.mx4_block(_block([1.0, math.inf])) == ([0] * 32, 255)
    assert experts.mx4_block(_block([math.nan])) == ([0] * 32, 255)


def test_mx4_is_the_nearest_value_by_fractions():
    """No value of the block's scale is nearer than the chosen one (exact rationals)."""
    rng = np.random.default_rng(3)
    X = (rng.standard_normal((8, 64)) * np.exp(3 * rng.standard_normal((8, 1)))).astype(np.float32).astype(float)
    codes, scales = experts.mx4_quantize(X)
    V = experts.mx4_values(codes, scales)
    for r in range(X.shape[0]):
        for k in range(X.shape[1]):
            unit = Fraction(2) ** (int(scales[r, k // 32]) - 127)
            err = abs(Fraction(X[r, k]) - Fraction(V[r, k]))
            for level in experts.MX4_LEVELS:
                for sign in (1, -1):
                    assert err <= abs(Fraction(X[r, k]) - sign * Fraction(level) * unit)
    assert np.array_equal(experts.mx4_quantize(V)[0], codes)   # values of the format stay


def test_mx4_packing():
    codes, scales = experts.mx4_quantize(np.array([_block([4.0, -1.0, 0.5])]))
    assert codes[0, 0] == (6 | 10 << 4) and codes[0, 1] == 1 and scales[0, 0] == 127
    assert list(experts.mx4_values(codes, scales)[0, :3]) == [4.0, -1.0, 0.5]


# ---------------------------------------------------------------- the C ABI on the host


@pytest.fixture(scope="module")
def lib():
    from sparse_gemm_b200 import build
    build.build()
    import sparse_gemm_b200 as sg
    return sg.library()


def _grouped(**kw):
    import sparse_gemm_b200 as sg
    return sg._GROUPED(kw.get("E", 4), kw.get("N", 64), kw.get("K", 64), kw.get("weight", 4096),
                       kw.get("status", 4096))


def _mx4(**kw):
    import sparse_gemm_b200 as sg
    return sg._MX4(kw.get("E", 1), kw.get("N", 64), kw.get("K", 64), kw.get("codes", 4096),
                   kw.get("scales", 4096), kw.get("status", 4096))


@pytest.mark.parametrize("bad,code", [(dict(E=0), 1), (dict(E=-1), 1), (dict(E=1025), 2), (dict(N=0), 1),
                                      (dict(N=60), 1), (dict(K=4), 1), (dict(K=0), 1), (dict(weight=0), 1),
                                      (dict(weight=4104), 1), (dict(status=0), 1), (dict(status=4098), 1)])
def test_bad_grouped_weight_is_refused(lib, bad, code):
    w = ctypes.byref(_grouped(**bad))
    assert lib.bsl_grouped_forward(4096, 8, 4096, w, None, 4096, 0, None) == code
    assert lib.bsl_grouped_backward_input(4096, 8, 4096, w, 4096, 0, None) == code
    assert lib.bsl_grouped_backward_weight(4096, 4096, 8, 4096, w, 4096, 4096, 1 << 30, None) == code
    assert lib.bsl_grouped_workspace_bytes(w) == 0


def test_bad_grouped_arguments_are_refused(lib):
    w = ctypes.byref(_grouped())
    for fn in (lambda x, t, o, y, b=None: lib.bsl_grouped_forward(x, t, o, w, b, y, 0, None),
               lambda x, t, o, y, b=None: lib.bsl_grouped_backward_input(x, t, o, w, y, 0, None)):
        assert fn(0, 8, 4096, 4096) == 1
        assert fn(4104, 8, 4096, 4096) == 1
        assert fn(4096, -1, 4096, 4096) == 1
        assert fn(4096, 8, 0, 4096) == 1
        assert fn(4096, 8, 4098, 4096) == 1
        assert fn(4096, 8, 4096, 0) == 1
        assert fn(0, 0, 4096, 0) == 0            # no row: nothing to do, no device needed
    assert lib.bsl_grouped_forward(4096, 8, 4096, w, 4104, 4096, 0, None) == 1
    assert lib.bsl_grouped_forward(4096, 8, 4096, None, None, 4096, 0, None) == 1
    dw = lambda dy, x, t, o, out, ws, n: lib.bsl_grouped_backward_weight(dy, x, t, o, w, out, ws, n, None)
    assert dw(0, 4096, 8, 4096, 4096, 4096, 1 << 30) == 1
    assert dw(4096, 0, 8, 4096, 4096, 4096, 1 << 30) == 1
    assert dw(4096, 4096, -1, 4096, 4096, 4096, 1 << 30) == 1
    assert dw(4096, 4096, 8, 0, 4096, 4096, 1 << 30) == 1
    assert dw(4096, 4096, 8, 4096, 0, 4096, 1 << 30) == 1
    need = lib.bsl_grouped_workspace_bytes(w)
    if need:
        assert dw(4096, 4096, 8, 4096, 4096, 0, need) == 1
        assert dw(4096, 4096, 8, 4096, 4096, 4096 + 16, need) == 1
        assert dw(4096, 4096, 8, 4096, 4096, 4096, need - 1) == 1
    db = lambda dy, t, o, E, N, out: lib.bsl_grouped_bias_grad(dy, t, o, E, N, out, None)
    assert [db(0, 8, 4096, 4, 64, 4096), db(4096, -1, 4096, 4, 64, 4096), db(4096, 8, 0, 4, 64, 4096),
            db(4096, 8, 4096, 0, 64, 4096), db(4096, 8, 4096, 4, 60, 4096), db(4096, 8, 4096, 4, 64, 0)] == [1] * 6
    assert db(4096, 8, 4096, 1025, 64, 4096) == 2
    assert lib.bsl_grouped_get_status(None, ctypes.byref(ctypes.c_int32()), None) == 1


@pytest.mark.parametrize("bad,code", [(dict(E=0), 1), (dict(E=1025), 2), (dict(N=0), 1), (dict(N=4), 1),
                                      (dict(K=48), 1), (dict(K=0), 1), (dict(codes=0), 1), (dict(codes=4104), 1),
                                      (dict(scales=0), 1), (dict(scales=4104), 1), (dict(status=0), 1)])
def test_bad_mx4_weight_is_refused(lib, bad, code):
    w = ctypes.byref(_mx4(**bad))
    assert lib.bsl_mx4_forward(4096, 4096, 8, w, None, 4096, None) == code
    assert lib.bsl_mx4_grouped_forward(4096, 4096, 8, 4096, w, None, 4096, 0, None) == code


def test_bad_mx4_arguments_are_refused(lib):
    w = ctypes.byref(_mx4())
    fwd = lambda c, s, m, y, b=None: lib.bsl_mx4_forward(c, s, m, w, b, y, None)
    assert [fwd(0, 4096, 8, 4096), fwd(4096, 0, 8, 4096), fwd(4096, 4096, -1, 4096), fwd(4096, 4096, 8, 0),
            fwd(4104, 4096, 8, 4096), fwd(4096, 4104, 8, 4096), fwd(4096, 4096, 8, 4096, 4104)] == [1] * 7
    assert fwd(0, 0, 0, 0) == 0
    assert lib.bsl_mx4_forward(4096, 4096, 8, ctypes.byref(_mx4(E=2)), None, 4096, None) == 1
    grp = lambda c, s, t, o, y, b=None: lib.bsl_mx4_grouped_forward(c, s, t, o, w, b, y, 0, None)
    assert [grp(0, 4096, 8, 4096, 4096), grp(4096, 0, 8, 4096, 4096), grp(4096, 4096, -1, 4096, 4096),
            grp(4096, 4096, 8, 0, 4096), grp(4096, 4096, 8, 4096, 0), grp(4096, 4096, 8, 4098, 4096)] == [1] * 6
    need = lib.bsl_mx4_workspace_bytes(8, w)
    assert need == 8 * (32 + 2) and lib.bsl_mx4_workspace_bytes(0, w) == 0
    lin = lambda x, t, o, y, ws, n, b=None, w=w: lib.bsl_mx4_linear(x, t, o, w, b, y, 0, ws, n, None)
    assert [lin(0, 8, None, 4096, 4096, need), lin(4096, -1, None, 4096, 4096, need), lin(4096, 8, None, 0, 4096, need),
            lin(4096, 8, None, 4096, 0, need), lin(4096, 8, None, 4096, 4104, need),
            lin(4096, 8, None, 4096, 4096, need - 1), lin(4096, 8, 4098, 4096, 4096, need),
            lin(4096, 8, None, 4096, 4096, need, 4104),
            lin(4096, 8, None, 4096, 4096, need, w=ctypes.byref(_mx4(E=2)))] == [1] * 9
    assert lin(0, 0, None, 0, 0, 0) == 0
    for fn in (lambda x, r, k, c, s: lib.bsl_mx4_quantize(x, r, k, c, s, None),
               lambda x, r, k, c, s: lib.bsl_mx4_dequantize(c, s, r, k, x, None)):
        assert [fn(0, 4, 64, 4096, 4096), fn(4096, -1, 64, 4096, 4096), fn(4096, 4, 48, 4096, 4096),
                fn(4096, 4, 0, 4096, 4096), fn(4096, 4, 64, 0, 4096), fn(4096, 4, 64, 4096, 0),
                fn(4104, 4, 64, 4096, 4096)] == [1] * 7
        assert fn(4096, 1 << 62, 64, 4096, 4096) == 2
        assert fn(0, 0, 64, 0, 0) == 0
    assert lib.bsl_mx4_get_status(None, ctypes.byref(ctypes.c_int32()), None) == 1


def test_sizes_past_the_index_range_are_refused(lib):
    """The kernels count rows and features in 32 bits up to the end of the last tile."""
    text = open(os.path.join(ROOT, "include", "bsl.h")).read()
    most = int(re.search(r"#define BSL_GROUPED_MAX_SIZE (\w+)", text).group(1), 16)
    big, P = 2 ** 31 - 32, 4096
    assert most + 2048 + 128 < 2 ** 31 and big > most
    for kw, T in (({}, most + 1), ({}, 2 ** 31 - 1), (dict(N=big), 8), (dict(K=big), 8)):
        w, q = ctypes.byref(_grouped(**kw)), ctypes.byref(_mx4(**kw))
        assert lib.bsl_grouped_forward(P, T, P, w, None, P, 0, None) == 2
        assert lib.bsl_grouped_backward_input(P, T, P, w, P, 0, None) == 2
        assert lib.bsl_grouped_backward_weight(P, P, T, P, w, P, P, 1 << 30, None) == 2
        assert lib.bsl_mx4_forward(P, P, T, q, None, P, None) == 2
        assert lib.bsl_mx4_grouped_forward(P, P, T, P, q, None, P, 0, None) == 2
        assert lib.bsl_mx4_linear(P, T, None, q, None, P, 0, P, 1 << 62, None) == 2
        if "K" not in kw:
            assert lib.bsl_grouped_bias_grad(P, T, P, 4, kw.get("N", 64), P, None) == 2


@pytest.mark.parametrize("name", ["_GROUPED", "_MX4"])
def test_binding_structs_match_the_header(name):
    import sparse_gemm_b200 as sg
    text = open(os.path.join(ROOT, "include", "bsl.h")).read()
    end = text.index("} bsl_" + name[1:].lower() + ";")
    body = re.sub(r"/\*.*?\*/", "", text[text.rindex("typedef struct {", 0, end):end], flags=re.S)
    assert [n for n, _ in getattr(sg, name)._fields_] == re.findall(r"\*?\s*(\w+)\s*[;,]", body)
    assert int(re.search(r"#define BSL_GROUPED_MAX_EXPERTS (\d+)", text).group(1)) == sg.GROUPED_MAX_EXPERTS


def test_cpu_tensors_and_wrong_types_are_refused():
    import torch
    import sparse_gemm_b200 as sg
    with pytest.raises(TypeError):
        sg.GroupedWeight(torch.zeros(2, 8, 8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        sg.quantize_mx4(torch.zeros(2, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        sg.quantize_mx4(None)
    with pytest.raises(TypeError):
        sg.Mx4Tensor(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8))
