"""State of the 4-bit modules: state_dict, moves between devices, casts, copies."""
import copy
import gc
import io

import numpy as np
import pytest
import torch

from tests._experts import normal, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


def layers(kind, bias=True):
    """Two modules of one kind with different weights, and a call of one on given rows."""
    rng = np.random.default_rng(41)
    lead = (3,) if kind == "grouped" else ()
    cls = sg.GroupedMx4Linear if kind == "grouped" else sg.Mx4Linear
    mods = [cls.from_dense(normal(rng, (*lead, 72, 96))[0], normal(rng, (*lead, 72))[0] if bias else None) for _ in range(2)]
    x = normal(rng, (20, 96))[0]
    off = offsets_of([9, 0, 11])[0]
    return mods, (lambda m: m(x, off)) if kind == "grouped" else (lambda m: m(x))


@pytest.mark.parametrize("kind", ["dense", "grouped"])
@pytest.mark.parametrize("bias", [True, False])
def test_state_dict_carries_the_weight(kind, bias):
    (a, b), call = layers(kind, bias)
    want, other = call(a), call(b)
    assert not torch.equal(want, other)
    state = a.state_dict()
    assert set(state) == {"codes", "scales"} | ({"bias"} if bias else set())
    buf = io.BytesIO()
    torch.save(state, buf)
    buf.seek(0)
    assert not b.load_state_dict(torch.load(buf)).missing_keys
    assert torch.equal(call(b), want)
    b.load_state_dict({k: v.clone() for k, v in state.items()}, assign=True)     # other storage
    assert torch.equal(call(b), want) and torch.equal(call(a), want)
    for key in state:
        with pytest.raises(RuntimeError, match=key):
            b.load_state_dict({k: v for k, v in state.items() if k != key})
        with pytest.raises(RuntimeError, match=key):
            b.load_state_dict({**state, key: state[key][:1]})
    assert torch.equal(call(b), want)


@pytest.mark.parametrize("kind", ["dense", "grouped"])
def test_moves_and_casts(kind):
    (a, b), call = layers(kind)
    want = call(a)
    for cast in ("float", "double", "bfloat16"):
        assert torch.equal(call(getattr(copy.deepcopy(a), cast)()), want)
    a.cpu()
    assert all(not t.is_cuda for t in a.state_dict().values())
    with pytest.raises(TypeError):
        call(a)
    a.cuda()
    assert torch.equal(call(a), want) and sg.mx4_status(a.weight4) == 0
    host = {k: v.cpu() for k, v in a.state_dict().items()}
    b.load_state_dict(host)
    assert torch.equal(call(b), want)


def test_memory_goes_with_the_module():
    gc.collect()
    before = torch.cuda.memory_allocated()
    mod = sg.Mx4Linear.from_dense(torch.randn(4096, 4096, device="cuda"))
    gc.collect()
    assert torch.cuda.memory_allocated() - before >= 4096 * 4096 * 17 // 32
    mod.cpu()
    gc.collect()
    assert torch.cuda.memory_allocated() == before


@pytest.mark.parametrize("kind", ["dense", "grouped"])
def test_handle_follows_the_buffers(kind):
    (a, b), call = layers(kind)
    wa, wb = call(a), call(b)
    q = a.weight4
    assert a.weight4 is q                        # kept while the buffers stay
    a.cuda()
    assert a.weight4 is q
    a.codes, a.scales = a.codes.clone(), a.scales.clone()
    assert a.weight4 is not q and torch.equal(call(a), wa)
    a.scales.sub_(1)                             # in place: half of every value
    c = copy.deepcopy(a)
    half = call(a)
    assert not torch.equal(half, wa) and torch.equal(call(c), half)
    a.weight4 = b.weight4
    a.bias.copy_(b.bias)
    assert torch.equal(call(a), wb) and torch.equal(call(c), half)


def test_old_pickles_open():
    """A module pickled when its weight was a plain attribute has the weight in its state."""
    (a, _), call = layers("dense")
    want = call(a)
    old = {**a.__dict__, "_buffers": {"bias": a.bias}, "weight4": a.weight4}
    del old["_weight4"]
    m = sg.Mx4Linear.__new__(sg.Mx4Linear)
    m.__setstate__(old)
    assert torch.equal(call(m), want) and set(m.state_dict()) == {"codes", "scales", "bias"}


def test_captured_module():
    (a, b), call = layers("grouped")
    call(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = call(a)
    a.load_state_dict(b.state_dict())            # in place: the next replay reads it
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, call(b))
