"""Chains of expert and 4-bit calls on one stream over few reused buffers.

Each kernel may be resident while its producer still writes, and a buffer that
a call reads was read with other contents a call or two before.  The chain
runs without a wait between its calls, eagerly and as a replayed graph, and
gives the bits of the same calls with a wait behind each.  Weights are made
anew inside it, too, just before they are used.
"""
import numpy as np
import pytest
import torch

from tests._experts import normal, offsets_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg

E, D = 3, 256      # experts, features in and out
STEPS = 6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


class Chain:
    def __init__(self, rows, seed):
        rng = np.random.default_rng(seed)
        self.off = offsets_of(rows)[0]
        T = sum(rows)
        w = lambda *s: normal(rng, s, D ** -0.5)[0]
        self.X = normal(rng, (T, D))[0]
        self.banks = [sg.quantize_mx4(w(E, D, D)) for _ in range(STEPS)]   # weights, a set for each step
        self.plain = [w(E, D, D) for _ in range(STEPS)]
        self.W = torch.zeros(E, D, D, dtype=torch.bfloat16, device="cuda")
        self.Wg = sg.GroupedWeight(self.W)
        self.Wq = sg.quantize_mx4(self.W)
        self.Wd = sg.quantize_mx4(w(D, D))
        self.bias = normal(rng, (E, D))[0]
        self.A, self.B = torch.empty_like(self.X), torch.empty_like(self.X)
        self.q = sg.quantize_mx4(self.X)
        self.dW = [torch.empty_like(self.W) for _ in range(STEPS)]
        self.db = [torch.empty_like(self.bias) for _ in range(STEPS)]
        self.Wq.status, self.Wd.status

    def results(self):
        return [self.A, self.B, *self.dW, *self.db]

    def poison(self):
        for t in (self.W, *self.results()):
            t.fill_(float("nan"))

    def run(self, wait=lambda: None):
        def did(_):
            wait()

        A, B, off = self.A, self.B, self.off
        did(sg.dequantize_mx4(self.q, out=A))
        for i in range(STEPS):
            did(sg.dequantize_mx4(self.banks[i], out=self.W))                        # a new weight ...
            did(sg.grouped_forward(A, self.Wg, off, bias=self.bias, out=B))          # ... read at once
            did(sg.quantize_mx4(self.plain[i], out=self.Wq))
            did(sg.grouped_forward_mx4(B, self.Wq, off, bias=self.bias, out=A))
            did(sg.grouped_bias_grad(A, off, out=self.db[i]))
            did(sg.grouped_backward_weight(A, B, self.Wg, off, out=self.dW[i]))
            did(sg.grouped_backward_input(A, self.Wg, off, out=B))
            did(sg.quantize_mx4(B, out=self.q))
            did(sg.forward_mx4(self.q, self.Wd, out=A))
            did(sg.forward_mx4(A, self.Wd, out=B))
            did(sg.dequantize_mx4(self.q, out=A))
            did(sg.grouped_forward(B, self.Wg, off, out=A))


@pytest.mark.parametrize("rows", [[1, 0, 2], [3, 0, 5], [9, 2, 5], [20, 0, 11], [70, 0, 90], [150, 300, 150]])
def test_chain_without_waits(rows):
    chain = Chain(rows, sum(rows))
    chain.poison()
    chain.run(torch.cuda.synchronize)
    want = [t.clone() for t in chain.results()]
    assert all(torch.isfinite(t.float()).all() for t in want)
    assert any(t.any() for t in want[2:])

    def same(tag):
        torch.cuda.synchronize()
        for i, (t, w) in enumerate(zip(chain.results(), want)):
            assert torch.equal(t, w), f"{tag}: result {i}"
        assert sg.grouped_status(chain.Wg) == 0 and sg.mx4_status(chain.Wq) == 0 and sg.mx4_status(chain.Wd) == 0

    for rep in range(5):
        chain.poison()
        sg.quantize_mx4(chain.X, out=chain.q)
        torch.cuda.synchronize()
        chain.run()
        same(f"eager {rep}")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        chain.run()
    torch.cuda.synchronize()
    for rep in range(5):
        chain.poison()
        sg.quantize_mx4(chain.X, out=chain.q)
        torch.cuda.synchronize()
        g.replay()
        same(f"replay {rep}")
