"""Pins of the oracles of the 8-bit layer, the router and the whole expert layer, host-side refusals of their entry
points (no GPU: every check precedes the first CUDA call), and source checks of their kernels."""
import ctypes
import glob
import itertools
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_gemm_b200", "csrc")


# ---------------------------------------------------------------- oracles


def levels():
    """The magnitudes of e4m3 and the parity of their codes, from the format: 2^-9 steps below 2^-6, then eight a binade."""
    out = [(Fraction(m, 512), m % 2) for m in range(8)]
    for e in range(-6, 9):
        out += [(Fraction(8 + m, 8) * Fraction(2) ** e, m % 2) for m in range(8)]
    return out[:-1]   # the last code is NaN


def test_e4m3_rounding_against_every_level():
    table = levels()
    assert len(table) == 127 and table[-1][0] == 448
    probes = set()
    for (a, _), (b, _) in zip(table, table[1:]):
        mid = (a + b) / 2
        probes |= {a, mid, mid * Fraction(4095, 4096), mid * Fraction(4097, 4096)}
    probes |= {Fraction(448), Fraction(460), Fraction(5000)}
    for p in sorted(probes):
        near = min(abs(p - v) for v, _ in table)
        best = [(v, odd) for v, odd in table if abs(p - v) == near]
        want = best[0][0] if len(best) == 1 else next(v for v, odd in best if not odd)
        for sign in (1, -1):
            assert experts.e4m3_nearest(np.array([sign * float(p)]))[0] == sign * float(want), p


def test_e4m3_rounding_against_torch():
    rng = np.random.default_rng(1)
    u = rng.standard_normal(20000) * np.exp2(rng.integers(-12, 9, 20000))
    u = np.clip(u.astype(np.float32), -448, 448)
    want = torch.from_numpy(u).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(experts.e4m3_nearest(u.astype(np.float64)), want)


def test_fp8_blocks_by_hand():
    X = np.zeros((130, 144))
    X[0, 0], X[0, 127], X[0, 128], X[129, 143], X[5, 140] = 448.0, -1.0, 3.0, 7.0, math.inf
    codes, scales = experts.fp8_quantize(X, 1)
    assert scales.shape == (130, 2) and scales[0, 0] == 1 and codes[0, 0] == 448 and codes[0, 127] == -1
    assert codes[0, 128] == 448 and scales[0, 1] == np.float32(3) / np.float32(448)
    assert np.isnan(scales[5, 1]) and not codes[5].any() and scales[7, 0] == np.float32(2.0 ** -100) / np.float32(448)
    codes, scales = experts.fp8_quantize(X, 128)
    assert scales.shape == (2, 2) and scales[0, 0] == 1 and np.isnan(scales[0, 1]) and codes[129, 143] == 448
    v = experts.fp8_values(codes, scales)
    assert v[0, 0] == 448 and np.isnan(v[3, 130]) and v[129, 143] == 448 * float(scales[1, 1])
    y, S = experts.fp8_product(np.ones((1, 144)), np.ones((1, 2)), np.ones((2, 144)), np.full((1, 2), 2.0))
    assert (y == 288).all() and (S == 288).all()


def test_route_against_all_choices():
    """The chosen are the best set under (logit, lower index), by trying every set; weights from the formula."""
    rng = np.random.default_rng(2)
    for trial in range(40):
        E, k = int(rng.integers(1, 7)), 1
        k = int(rng.integers(1, E + 1))
        row = rng.integers(-2, 3, E).astype(float)
        e, w, offsets, order = experts.route(row[None], k, renormalize=False)
        want = max(itertools.permutations(range(E), k), key=lambda s: [(row[i], -i) for i in s])
        assert tuple(e[0]) == want
        p = np.exp(row) / np.exp(row).sum()
        assert np.allclose(w[0], p[list(want)], rtol=1e-14)
        assert list(order) == sorted(range(k), key=lambda j: e[0][j]) and list(offsets) == [sum(x < i for x in want) for i in range(E + 1)]


def test_route_gradient_against_torch():
    rng = np.random.default_rng(3)
    for score, renormalize in itertools.product(("softmax", "sigmoid"), (False, True)):
        f = rng.standard_normal((5, 9))
        l = torch.from_numpy(f).requires_grad_(True)
        e, w, _, _ = experts.route(f, 3, score, renormalize, 1.5)
        s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        p = torch.gather(s, 1, torch.from_numpy(e))
        mine = 1.5 * (p / p.sum(1, keepdim=True) if renormalize else p)
        assert np.allclose(mine.detach().numpy(), w, rtol=1e-12)
        g = rng.standard_normal((5, 3))
        (mine * torch.from_numpy(g)).sum().backward()
        got, S = experts.route_backward(g, f, e, score, renormalize, 1.5)
        assert np.allclose(got, l.grad.numpy(), rtol=1e-10, atol=1e-13) and (np.abs(got) <= S * (1 + 1e-9) + 1e-15).all()


def test_moe_against_grouped_products():
    rng = np.random.default_rng(4)
    T, E, k, H, I = 4, 3, 2, 5, 6
    X, W13, W2 = rng.standard_normal((T, H)), rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    e = np.array([[0, 2], [1, 0], [2, 2], [7, 1]])
    w = rng.standard_normal((T, k))
    got, B = experts.moe_forward(X, W13, W2, e, w)
    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if e[t, j] < E:
                z, _ = experts.grouped_forward(X[t:t + 1], W13[e[t, j]:e[t, j] + 1], [0, 1])
                h = torch.nn.functional.silu(torch.from_numpy(z[:, :I])).numpy() * z[:, I:]
                want[t] += w[t, j] * experts.grouped_forward(h, W2[e[t, j]:e[t, j] + 1], [0, 1])[0][0]
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12) and (B > 0).all()


# ---------------------------------------------------------------- the C ABI on the host


@pytest.fixture(scope="module")
def lib():
    from sparse_gemm_b200 import build
    build.build()
    import sparse_gemm_b200 as sg
    return sg.library()


def _fp8(**kw):
    import sparse_gemm_b200 as sg
    return sg._FP8(kw.get("E", 1), kw.get("N", 64), kw.get("K", 64), kw.get("codes", 4096), kw.get("scales", 4096),
                   kw.get("status", 4096))


def _grouped(**kw):
    import sparse_gemm_b200 as sg
    return sg._GROUPED(kw.get("E", 4), kw.get("N", 64), kw.get("K", 64), kw.get("weight", 4096), kw.get("status", 4096))


P = 4096


@pytest.mark.parametrize("bad,code", [(dict(E=0), 1), (dict(E=1025), 2), (dict(N=0), 1), (dict(N=4), 1), (dict(K=24), 1),
                                      (dict(K=0), 1), (dict(codes=0), 1), (dict(codes=4104), 1), (dict(scales=0), 1),
                                      (dict(scales=4104), 1), (dict(status=0), 1), (dict(K=2 ** 31 - 16), 2)])
def test_bad_fp8_weight_is_refused(lib, bad, code):
    w = ctypes.byref(_fp8(**bad))
    assert lib.bsl_fp8_product(P, P, 8, P, w, 0, None, P, 0, None) == code
    assert lib.bsl_fp8_linear(P, 8, P, w, 0, None, P, 0, P, 1 << 40, None) == code
    assert lib.bsl_fp8_workspace_bytes(8, w, 0) == 0
    assert lib.bsl_moe_forward_fp8(P, 1, P, P, 1, w, w, P, P, 1 << 40, None) == code


def test_bad_fp8_arguments_are_refused(lib):
    w = ctypes.byref(_fp8())
    prod = lambda c, s, t, o, y, tr=0, b=None, w=w: lib.bsl_fp8_product(c, s, t, o, w, tr, b, y, 0, None)
    for tr in (0, 1):
        assert [prod(0, P, 8, P, P, tr), prod(P, 0, 8, P, P, tr), prod(P, P, -1, P, P, tr), prod(P, P, 8, P, 0, tr),
                prod(P + 8, P, 8, P, P, tr), prod(P, P + 8, 8, P, P, tr), prod(P, P, 8, P + 2, P, tr)] == [1] * 7
        assert prod(P, P, 8, None, P, tr, w=ctypes.byref(_fp8(E=2))) == 1       # several experts without offsets
        assert prod(P, P, 2 ** 31 - 1, P, P, tr) == 2
        assert prod(0, 0, 0, None, 0, tr) == 0
    assert prod(P, P, 8, P, P, 0, P + 8) == 1                                   # misaligned bias
    assert prod(P, P, 8, P, P, 1, P) == 1                                       # the gradient has no bias
    assert prod(P, P, 8, P, P, 1, w=ctypes.byref(_fp8(N=72))) == 1              # rows of 72 codes
    need = lib.bsl_fp8_workspace_bytes(8, w, 0)
    assert need == 8 * (64 + 4) and lib.bsl_fp8_workspace_bytes(0, w, 0) == 0
    assert lib.bsl_fp8_workspace_bytes(8, ctypes.byref(_fp8(N=272)), 1) == 8 * (272 + 12)
    lin = lambda x, t, o, y, ws, n, tr=0, b=None: lib.bsl_fp8_linear(x, t, o, w, tr, b, y, 0, ws, n, None)
    assert [lin(0, 8, None, P, P, need), lin(P, -1, None, P, P, need), lin(P, 8, None, 0, P, need), lin(P, 8, None, P, 0, need),
            lin(P, 8, None, P, P + 8, need), lin(P, 8, None, P, P, need - 1), lin(P, 8, P + 2, P, P, need),
            lin(P, 8, None, P, P, need, 0, P + 8)] == [1] * 8
    assert lin(0, 0, None, 0, 0, 0) == 0
    for fn in (lambda x, p, r, k, b, c, s: lib.bsl_fp8_quantize(x, p, r, k, b, c, s, None),
               lambda x, p, r, k, b, c, s: lib.bsl_fp8_dequantize(c, s, p, r, k, b, x, None)):
        assert [fn(0, 1, 4, 64, 1, P, P), fn(P, -1, 4, 64, 1, P, P), fn(P, 1, -1, 64, 1, P, P), fn(P, 1, 4, 40, 1, P, P),
                fn(P, 1, 4, 0, 1, P, P), fn(P, 1, 4, 64, 2, P, P), fn(P, 1, 4, 64, 1, 0, P), fn(P, 1, 4, 64, 1, P, 0),
                fn(P + 8, 1, 4, 64, 128, P, P)] == [1] * 9
        assert fn(P, 1 << 31, 1 << 40, 64, 1, P, P) == 2
        assert fn(0, 1, 0, 64, 1, 0, 0) == 0 and fn(0, 0, 4, 64, 128, 0, 0) == 0
    assert lib.bsl_fp8_get_status(None, ctypes.byref(ctypes.c_int32()), None) == 1


def test_bad_route_arguments_are_refused(lib):
    rt = lambda l=P, ty=0, T=4, E=8, k=2, s=0, e=P, w=P, off=P, order=P, ws=None, n=0: \
        lib.bsl_route(l, ty, T, E, k, s, 1, 1.0, e, w, off, order, ws, n, None)
    assert [rt(l=0), rt(l=P + 2), rt(ty=2), rt(T=-1), rt(E=0), rt(k=0), rt(k=9), rt(s=2), rt(e=0), rt(w=0), rt(off=0), rt(order=0),
            rt(off=P + 2), rt(l=P + 1, ty=1)] == [1] * 14
    assert [rt(E=1025), rt(E=64, k=33), rt(T=2 ** 30, k=4)] == [2] * 3
    need = lib.bsl_route_workspace_bytes(1000, 8, 2)
    assert need > 0 and lib.bsl_route_workspace_bytes(100, 8, 2) == 0 and lib.bsl_route_workspace_bytes(1000, 8, 9) == 0
    assert [rt(T=1000), rt(T=1000, ws=P, n=need - 1), rt(T=1000, ws=P + 2, n=need)] == [1] * 3
    assert rt(T=0, l=0, e=0, w=0, off=None, order=None) == 0
    bw = lambda d=P, l=P, ty=0, T=4, E=8, k=2, e=P, s=0, out=P: lib.bsl_route_backward(d, l, ty, T, E, k, e, s, 1, 1.0, out, None)
    assert [bw(d=0), bw(l=0), bw(ty=3), bw(T=-1), bw(k=9), bw(e=0), bw(s=5), bw(out=0), bw(out=P + 2), bw(d=P + 2)] == [1] * 10
    assert bw(E=1025) == 2 and bw(T=0, d=0, l=0, e=0, out=0) == 0


def test_bad_moe_arguments_are_refused(lib):
    pairs = {"bsl_moe_forward": (_grouped(N=128, K=48), _grouped(N=48, K=64)),
             "bsl_moe_forward_fp8": (_fp8(E=4, N=128, K=48), _fp8(E=4, N=48, K=64))}
    for name, (w13, w2) in pairs.items():
        need = lib.bsl_moe_workspace_bytes(3, 2, 64)
        assert need == 3 * 2 * 64 * 2
        fn = lambda x=P, T=3, e=P, w=P, k=2, a=w13, b=w2, y=P, ws=P, n=need: getattr(lib, name)(
            x, T, e, w, k, ctypes.byref(a), ctypes.byref(b), y, ws, n, None)
        assert [fn(x=0), fn(x=P + 8), fn(T=-1), fn(e=0), fn(e=P + 2), fn(w=0), fn(k=0), fn(y=0), fn(ws=0), fn(ws=P + 8), fn(n=need - 1),
                fn(a=w2, b=w13), fn(b=w13)] == [1] * 13
        assert fn(T=65, n=1 << 30) == 2 and fn(k=33, n=1 << 30) == 2
        assert fn(x=0, T=0, e=0, w=0, y=0, ws=0, n=0) == 0
        other = type(w2)(5, w2.N, w2.K, P, *((P, P) if "fp8" in name else (P,)))
        assert fn(b=other) == 1                                                 # another number of experts
    assert lib.bsl_moe_workspace_bytes(0, 2, 64) == 0


def test_moe_refuses_more_units_than_it_counts(lib):
    """Tokens x choices x I / 8 units of work are counted in 32 bits."""
    wide = 2 ** 23 + 16   # 64 x 32 x 2^20 = 2^31 units and more
    for name, make in (("bsl_moe_forward", _grouped), ("bsl_moe_forward_fp8", _fp8)):
        shape = {} if make is _grouped else {"E": 4}
        w13, w2 = make(N=2 * wide, K=16, **shape), make(N=16, K=wide, **shape)
        assert getattr(lib, name)(P, 64, P, P, 32, ctypes.byref(w13), ctypes.byref(w2), P, P, 1 << 50, None) == 2


@pytest.mark.parametrize("T,E,k", [(129, 8, 2), (16384, 128, 8), (131072, 128, 8), (131073, 128, 32), (1 << 20, 128, 8), (1 << 23, 16, 1)])
def test_the_sorts_counts_grow_with_the_tokens(lib, T, E, k):
    """Every CTA of the sort reads the counts of all runs: their number stays small, whatever the tokens, as long as a
    run's pairs (8192 at most) fit in shared memory."""
    runs = lib.bsl_route_workspace_bytes(T, E, k) // (4 * E)
    assert 0 < runs <= max(1024, -(-T // (8192 // k)))


def test_the_binding_matches_the_header():
    import sparse_gemm_b200 as sg
    text = open(os.path.join(ROOT, "include", "bsl.h")).read()
    end = text.index("} bsl_fp8;")
    body = re.sub(r"/\*.*?\*/", "", text[text.rindex("typedef struct {", 0, end):end], flags=re.S)
    assert [n for n, _ in sg._FP8._fields_] == re.findall(r"\*?\s*(\w+)\s*[;,]", body)
    for name, value in (("BSL_ROUTE_MAX_K", sg.ROUTE_MAX_K), ("BSL_MOE_MAX_TOKENS", sg.MOE_MAX_TOKENS)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value


def test_cpu_tensors_and_wrong_types_are_refused():
    import sparse_gemm_b200 as sg
    X = torch.zeros(2, 64, dtype=torch.bfloat16)
    for bad in (lambda: sg.quantize_fp8(X), lambda: sg.quantize_fp8(None), lambda: sg.route(torch.zeros(2, 8), 2),
                lambda: sg.Fp8Tensor(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1)), lambda: sg.Fp8Tensor(None, None),
                lambda: sg.moe_forward(X, None, None, None, None), lambda: sg.route(None, 2)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        sg.forward_fp8(X, X)


# ---------------------------------------------------------------- sources

FILES = sorted(os.path.basename(p) for pattern in ("fp8*", "route*", "moe*", "ring*") for p in glob.glob(os.path.join(CSRC, pattern)))


def code_of(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_the_kernels_are_looked_at():
    assert {"fp8.cu", "fp8_few.cu", "fp8_quant.cu", "moe.cu", "ring.cuh", "route.cu"} <= set(FILES)
    assert all("wait_for_prior_grid()" in code_of(f) for f in FILES if "__global__" in code_of(f))


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads_in_dependent_kernels(name):
    """Each kernel is resident before the one that writes its inputs has ended."""
    assert not re.findall(r"__ldg\w*\s*\(|ld\.global\.nc[\w.:]*|__restrict__", code_of(name))


def test_kernels_before_early_readers_let_them_start_late():
    """k_moe_down reads choices and weights, and the products of few rows weights and offsets, before they wait for the
    kernel before: that one lets its dependents start only behind its own wait, so what it waited for has ended."""
    for name, kernel in (("moe.cu", "k_moe_up(const MoeArgs"), ("fp8_quant.cu", "k_fp8_quantize_rows(const Fp8Args")):
        code = code_of(name)
        body = code[code.index(kernel):]
        assert body.index("wait_for_prior_grid()") < body.index("dependents_may_launch()"), name
    code = code_of("moe.cu")
    run = code[code.index("bsl_status run(const MoeArgs"):]
    assert run.index("k_moe_up<F8, NT>, static_cast") < run.index("launch_dependent_cluster(k_moe_down")
