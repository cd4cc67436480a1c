"""A weight that is quantised anew into the same tensors right before it is used. The product's kernel may read the
weight and its scales ahead of the kernel in front of it (the quantisation of x), never ahead of the work before that.
"""
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from fp8_testlib import BF, E4, F32, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()
    yield
    assert dw.dora_device_status() == 0, "a kernel's bounded wait ran out"


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("T", [1, 20, 37, 100, 200, 2100])
@pytest.mark.parametrize("d_out,d_in", [(272, 400), (1040, 2064), (4096, 4096)])
def test_requantised_right_before_each_call(d_out, d_in, T, odd, backward):
    """odd: the scales are also multiplied in place, so that they are no powers of two."""
    fn = dw.dora_fp8_backward if backward else dw.dora_fp8_forward
    x = torch.randn(T, d_out if backward else d_in, generator=gen(1), device="cuda").to(BF)
    Ws = [torch.randn(d_out, d_in, generator=gen(2 + i), device="cuda") * 4.0 ** -i for i in range(4)]
    wq = torch.zeros(d_out, d_in, dtype=E4, device="cuda")
    ws = torch.zeros(-(-d_out // 128), -(-d_in // 128), device="cuda")

    def run(wait):
        ys = []
        for i in range(24):
            dw.dora_fp8_quantize(Ws[i % 4], block="tile", q=wq, scale=ws)
            if odd:
                ws.mul_(1.25)
            if wait:
                torch.cuda.synchronize()
            ys.append(fn(x, wq, ws, out_dtype=F32))
            if wait:
                torch.cuda.synchronize()
        return ys

    ref, got = run(True), run(False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    y = [None] * 8
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(8):
            dw.dora_fp8_quantize(Ws[i % 4], block="tile", q=wq, scale=ws)
            if odd:
                ws.mul_(1.25)
            y[i] = fn(x, wq, ws, out_dtype=F32)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, y))
