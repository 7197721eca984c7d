"""Outputs that overlap any input of an expert or 4-bit call are refused: the rows, the weight and, in
buffers of their own, scales, bias and offsets."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_gemm_b200 as sg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_gemm_b200 import build
    build.build()


T, N, K, E = 8, 32, 64, 2


class Case:
    def __init__(self):
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
        self.X, self.dY = bf(T, K), bf(T, N)
        self.Wg = sg.GroupedWeight(bf(E, N, K))
        # one buffer of 16-byte pieces that inputs and outputs are cut from
        self.buf = bf(8192)
        self.offsets = self.buf[:2 * (E + 1)].view(torch.int32)            # bytes 0 .. 11
        self.bias = self.buf[64:64 + E * N].view(E, N)                     # bytes 128 .. 255
        self.off = torch.tensor([0, 3, T], dtype=torch.int32, device="cuda")

    def cut(self, at, *shape):
        """A bf16 view of the buffer that begins `at` bytes into it."""
        n = 1
        for d in shape:
            n *= d
        return self.buf[at // 2:at // 2 + n].view(*shape)


def refused(call):
    with pytest.raises(ValueError, match="overlap"):
        call()


def test_bias_and_offsets_of_the_expert_calls():
    c = Case()
    refused(lambda: sg.grouped_forward(c.X, c.Wg, c.offsets, out=c.cut(0, T, N)))
    refused(lambda: sg.grouped_forward(c.X, c.Wg, c.off, bias=c.bias, out=c.cut(0, T, N)))
    refused(lambda: sg.grouped_forward(c.X, c.Wg, c.off, bias=c.bias, out=c.cut(240, T, N)))
    refused(lambda: sg.grouped_backward_input(c.dY, c.Wg, c.offsets, out=c.cut(0, T, K)))
    refused(lambda: sg.grouped_backward_weight(c.dY, c.X, c.Wg, c.offsets, out=c.cut(0, E, N, K)))
    refused(lambda: sg.grouped_bias_grad(c.dY, c.offsets, out=c.cut(0, E, N)))
    # neighbours are fine
    sg.grouped_forward(c.X, c.Wg, c.off, bias=c.bias, out=c.cut(256, T, N))
    sg.grouped_bias_grad(c.dY, c.offsets, out=c.cut(16, E, N))
    assert sg.grouped_status(c.Wg) == 0


def scattered(rows, K, c, at):
    """A 4-bit tensor whose scales lie `at` bytes into the case's buffer, apart from its codes."""
    scales = c.buf.view(torch.uint8)[at:at + rows * K // 32].view(rows, K // 32)
    return sg.Mx4Tensor(torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda"), scales)


def test_separately_held_scales():
    c = Case()
    w, x = scattered(N, K, c, 1024), scattered(T, K, c, 2048)              # 64 and 16 bytes
    other_w = sg.quantize_mx4(c.Wg.weight[0].contiguous())
    for at, refuse in ((512, False), (528, True), (1072, True), (1088, False)):
        call = lambda: sg.forward_mx4(c.X, w, out=c.cut(at, T, N))
        refused(call) if refuse else call()
    for at, refuse in ((1536, False), (1552, True), (2048, True), (2064, False)):
        call = lambda: sg.forward_mx4(x, other_w, out=c.cut(at, T, N))
        refused(call) if refuse else call()
    for at, refuse in ((1024, False), (1040, True), (2048, True), (2064, False)):
        call = lambda: sg.dequantize_mx4(x, out=c.cut(at, T, K))
        refused(call) if refuse else call()
    w3 = sg.Mx4Tensor(torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda"),
                      c.buf.view(torch.uint8)[4096:4096 + E * N * 2].view(E, N, 2))
    refused(lambda: sg.grouped_forward_mx4(c.X, w3, c.off, out=c.cut(4096, T, N)))
    refused(lambda: sg.grouped_forward_mx4(c.X, w3, c.offsets, out=c.cut(0, T, N)))
    refused(lambda: sg.grouped_forward_mx4(c.X, w3, c.off, bias=c.bias, out=c.cut(0, T, N)))
    refused(lambda: sg.forward_mx4(c.X, other_w, bias=c.bias.view(-1)[:N], out=c.cut(144, T, N)))
    assert sg.mx4_status(w) == 0 and sg.mx4_status(w3) == 0


def test_quantise_into_its_own_input():
    c = Case()
    X = c.cut(1024, T, K)                                                  # bytes 1024 .. 2047
    flat = c.buf.view(torch.uint8)
    codes = lambda at: flat[at:at + T * K // 2].view(T, K // 2)            # 256 bytes
    scales = lambda at: flat[at:at + T * K // 32].view(T, K // 32)         # 16 bytes
    for a, b, refuse in ((1024, 0, True), (1792, 0, True), (512, 1024, True), (512, 2032, True), (784, 0, True),
                         (768, 2048, False), (2048, 1008, False)):
        q = sg.Mx4Tensor(codes(a), scales(b))
        call = lambda: sg.quantize_mx4(X, out=q)
        refused(call) if refuse else call()
