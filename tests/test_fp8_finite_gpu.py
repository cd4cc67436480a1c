"""The 8-bit products of few tokens on weights and operands without a NaN, so that every shape is held to the bound on
the whole matrix. Scales that are no powers of two are folded in fp32 in every CTA, and held to the fold's own bound.
"""
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from fp8_testlib import BF, E4, E5, F32, blocks, call, check, codes, gen, scales, wide_rows, wide_tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()
    yield
    assert dw.dora_device_status() == 0, "a kernel's bounded wait ran out"


SHAPES = [(1, 16, 16), (1, 272, 1040), (5, 1040, 272), (16, 384, 640), (17, 144, 4112), (33, 528, 128), (64, 2048, 256),
          (65, 128, 2064), (100, 400, 400), (128, 128, 128), (129, 272, 272), (257, 528, 912), (300, 16, 656), (512, 1296, 336),
          (700, 640, 2048), (8, 272, 8208), (48, 272, 40976)]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("T,d_out,d_in", SHAPES)
def test_products_of_given_codes(T, d_out, d_in, out_dtype, powers, fp8, backward):
    K = d_out if backward else d_in
    wq, ws = codes(d_out, d_in, E4, 1), scales(blocks(d_out), blocks(d_in), 2, powers, -3, 4)
    xq, xs = codes(T, K, fp8, 3), scales(blocks(K), T, 4, powers)
    w = wide_tiles(wq, ws)
    check(call(backward, xq, wq, ws, xs, out_dtype=out_dtype), wide_rows(xq, xs), w if backward else w.T, K, whole=powers)


@pytest.mark.parametrize("T", [1, 24, 200])
def test_two_calls_at_once(T):
    """Calls on two streams share nothing."""
    wq, ws = codes(1040, 1168, E4, 5), scales(9, 10, 6, False)
    xs = [torch.randn(T, 1168, generator=gen(7 + i), device="cuda").to(BF) for i in range(2)]
    ref = [call(False, x, wq, ws) for x in xs]
    assert all(bool(torch.isfinite(r).all()) for r in ref)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(20):
        for o, x, st in zip(outs, xs, streams):
            o.append(call(False, x, wq, ws, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(v, r) for r, o in zip(ref, outs) for v in o)
