"""The 8-bit products at the sizes that go to the kernel of CTA pairs (256 x 256 tiles), and the quantiser at the sizes
that go to its form with eight loads per thread, against float64. Every product test asserts, by the kernel's
name in the library's own timing records, that its call gets there.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from fp8_testlib import BF, E4, E5, F32, NAME, blocks, call, check, codes, gen, launches, scales, wide_rows, wide_tiles
from oracle import fp8 as of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()
    yield
    assert dw.dora_device_status() == 0, "a kernel's bounded wait ran out"


# T, results per token N, sum length K: partial tiles in T, in N (a whole 128 columns and a piece, or a piece alone, of the
# last 256) and in K; one to more than two rounds of the six stages; K beyond what an fp32 result adds in one accumulator
SHAPES = [(2100, 2464, 1040), (2100, 2320, 2064), (270, 27664, 784), (140, 20016, 272), (200, 20112, 128), (4100, 1168, 144),
          (1300, 4112, 4240)]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_products_of_given_codes(T, N, K, out_dtype, powers, fp8, backward):
    wq = codes(K, N, E4, 1) if backward else codes(N, K, E4, 1)
    ws = scales(blocks(wq.shape[0]), blocks(wq.shape[1]), 2, powers, -3, 4)
    xq, xs = codes(T, K, fp8, 3), scales(blocks(K), T, 4, powers)
    buf = torch.full((T + 3, N), 7.0, dtype=out_dtype, device="cuda")
    names = launches(lambda: call(backward, xq, wq, ws, xs, out_dtype=out_dtype))
    assert names[-1] == ("fp8_backward_pairs" if backward else "fp8_forward_pairs"), names
    out = call(backward, xq, wq, ws, xs, out=buf[:T])
    w = wide_tiles(wq, ws)
    check(out, wide_rows(xq, xs), w if backward else w.T, K, whole=powers and (out_dtype == BF or blocks(K) <= 32))
    assert bool((buf[T:] == 7).all())


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("T,N,K", [(2100, 2464, 1040), (270, 27664, 784), (1300, 4112, 4240)])
def test_products_of_wide_operands(T, N, K, fp8, dtype, backward):
    """Quantised in the call: the product of the oracle's codes, and the bits of the two-call form."""
    x = (torch.randn(T, K, generator=gen(5), device="cuda") *
         torch.exp2(torch.randint(-12, 12, (T, blocks(K)), generator=gen(6), device="cuda").float()).repeat_interleave(128, 1)[:, :K]).to(dtype)
    w = torch.randn(*((K, N) if backward else (N, K)), generator=gen(7), device="cuda") * 0.05
    wq, ws = dw.dora_fp8_quantize(w, block="tile")
    assert launches(lambda: call(backward, x, wq, ws, fp8_dtype=fp8)) == \
        ["fp8_quantize_rows", "fp8_backward_pairs" if backward else "fp8_forward_pairs"]
    out = call(backward, x, wq, ws, fp8_dtype=fp8)
    q, s = of.quantize(x.float().cpu().numpy().astype(np.float64), NAME[fp8], False)
    xq, xs = dw.dora_fp8_quantize(x, dtype=fp8)
    assert np.array_equal(xq.float().cpu().numpy(), q) and np.array_equal(xs.cpu().numpy(), s)
    ww = wide_tiles(wq, ws)
    check(out, torch.from_numpy(of.widen_rows(q, s)).cuda(), ww if backward else ww.T, K, whole=dtype == BF or blocks(K) <= 32)
    assert torch.equal(out, call(backward, xq, wq, ws, xs, out_dtype=dtype))


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("which,value", [("w", 1.5), ("w", 0.0), ("w", -2.0), ("w", 1e-40), ("x", 0.7), ("x", 0.0), ("x", -1.0)])
@pytest.mark.parametrize("at", [0, -1, 0.37])
def test_one_scale_that_is_no_power_of_two(at, which, value, backward):
    """Among powers of two, wherever it lies: the whole call is then folded, and held to the fold's bound."""
    T, N, K = 2100, 2464, 1040
    wq = codes(K, N, E4, 11) if backward else codes(N, K, E4, 11)
    ws, xs = scales(blocks(wq.shape[0]), blocks(wq.shape[1]), 12, True, -3, 4), scales(blocks(K), T, 14, True)
    xq = codes(T, K, E4, 13)
    s = (ws if which == "w" else xs).view(-1)
    s[int(at * s.numel()) if isinstance(at, float) else at] = value
    assert launches(lambda: call(backward, xq, wq, ws, xs, out_dtype=F32))[-1].endswith("_pairs")
    w = wide_tiles(wq, ws)
    check(call(backward, xq, wq, ws, xs, out_dtype=F32), wide_rows(xq, xs), w if backward else w.T, K, whole=False)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("given", [True, False])
def test_rows_that_are_not_finite_stay_in_their_rows(given, powers, backward):
    T, N, K = 2100, 2464, 1040
    wq = codes(K, N, E4, 21) if backward else codes(N, K, E4, 21)
    ws = scales(blocks(wq.shape[0]), blocks(wq.shape[1]), 22, powers, -3, 4)
    x = torch.randn(T, K, generator=gen(23), device="cuda").to(BF)
    run = lambda v: call(backward, *([v, wq, ws] if not given else [dw.dora_fp8_quantize(v)[0], wq, ws, dw.dora_fp8_quantize(v)[1]]))
    assert launches(lambda: run(x))[-1].endswith("_pairs")
    clean = run(x)
    bad = [0, 127, 128, 300, 1023, T - 1]
    for i, v in zip(bad, (float("inf"), float("nan"), float("-inf"), float("nan"), float("inf"), float("nan"))):
        x[i, (i * 7) % K] = v
    out = run(x)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert not torch.isfinite(out[bad]).any() and bool(torch.isfinite(clean).all())
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("T,N", [(2100, 2464), (20, 272), (100, 528), (8, 272)])
def test_codes_that_are_nan(T, N, powers):
    """A NaN among x's codes makes its row NaN, one among the weight's its column; the rest is as without them."""
    K = 1040
    wq, xq = codes(N, K, E4, 31), codes(T, K, E4, 32)
    ws, xs = scales(blocks(N), blocks(K), 33, powers, -3, 4), scales(blocks(K), T, 34, powers)
    clean = call(False, xq, wq, ws, xs, out_dtype=F32)
    assert T < 2000 or launches(lambda: call(False, xq, wq, ws, xs, out_dtype=F32))[-1].endswith("_pairs")
    for q, i in ((xq, 0), (xq, T - 2), (wq, 5), (wq, N - 1)):
        q.view(torch.uint8)[i, (i * 11) % K] = 0x7F
    out = call(False, xq, wq, ws, xs, out_dtype=F32)
    rows, cols = torch.zeros(T, 1, dtype=torch.bool, device="cuda"), torch.zeros(1, N, dtype=torch.bool, device="cuda")
    rows[[0, T - 2]], cols[:, [5, N - 1]] = True, True
    assert torch.equal(torch.isnan(out), rows | cols) and bool(torch.isfinite(clean).all())
    assert torch.equal(out[~(rows | cols)], clean[~(rows | cols)])


def test_zero_rows_and_zero_scales():
    T, N, K = 2100, 2464, 528
    wq, x = codes(N, K, E4, 41), torch.randn(T, K, generator=gen(42), device="cuda").to(BF)
    x[1200] = 0
    for powers in (True, False):
        ws = scales(blocks(N), blocks(K), 43, powers, -3, 4)
        assert launches(lambda: call(False, x, wq, ws))[-1].endswith("_pairs")
        y = call(False, x, wq, ws)
        assert bool((y[1200] == 0).all()) and bool((y[:1200] != 0).any())
    ws[3] = 0
    y = call(False, x, wq, ws)
    assert bool((y[:, 384:512] == 0).all()) and bool((y[:1200, :384] != 0).any())


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("powers", [True, False])
def test_captured_and_on_two_streams(powers, backward):
    T, N, K = 2100, 2464, 1040
    wq = codes(K, N, E4, 51) if backward else codes(N, K, E4, 51)
    ws = scales(blocks(wq.shape[0]), blocks(wq.shape[1]), 52, powers, -3, 4)
    xs = [torch.randn(T, K, generator=gen(53 + i), device="cuda").to(BF) for i in range(2)]
    ref = [call(backward, x, wq, ws) for x in xs]
    assert launches(lambda: call(backward, xs[0], wq, ws))[-1].endswith("_pairs")
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(10):
        for o, x, st in zip(outs, xs, streams):
            o.append(call(backward, x, wq, ws, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(v, r) for r, o in zip(ref, outs) for v in o)
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(backward, x, wq, ws)
        z = call(backward, x, wq, ws)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref[i]) and torch.equal(z, ref[i])


@pytest.mark.parametrize("backward", [False, True])
def test_a_padded_batch(backward):
    T, N, K = 2100, 2464, 1040
    wq = codes(K, N, E4, 61) if backward else codes(N, K, E4, 61)
    ws = scales(blocks(wq.shape[0]), blocks(wq.shape[1]), 62, True, -3, 4)
    x = torch.full((T + 200, K), float("nan"), dtype=BF, device="cuda")
    x[:T] = torch.randn(T, K, generator=gen(63), device="cuda")
    out = torch.full((T + 200, N), 7.0, dtype=BF, device="cuda")
    assert launches(lambda: call(backward, x[:T], wq, ws))[-1].endswith("_pairs")
    call(backward, x[:T], wq, ws, out=out[:T])
    assert bool(torch.isfinite(out[:T]).all()) and bool((out[T:] == 7).all())
    assert torch.equal(out[:T], call(backward, x[:T].clone(), wq, ws))


@pytest.mark.parametrize("K", [400, 2320])
def test_gradient_by_differences(K):
    """dx = dy W is the derivative of sum(dy y) along any direction (small whole numbers: exact codes). With K = 400 the
    gradient comes from the kernel for few tiles, with 2320 both directions run on pairs."""
    T, N = 2100, 2464
    rng = np.random.default_rng(9)
    whole = lambda lo, hi, *shape: torch.from_numpy(rng.integers(lo, hi, shape).astype(np.float32)).cuda()
    wq, ws = codes(N, K, E4, 71), scales(blocks(N), blocks(K), 72, True, -3, 4)
    x0, step, dy = whole(-8, 9, T, K), whole(-7, 8, T, K), whole(-8, 9, T, N)
    f = lambda x: float((call(False, x, wq, ws).double() * dy.double()).sum())
    diff = f(x0 + step) - f(x0)
    assert launches(lambda: call(False, x0, wq, ws))[-1] == "fp8_forward_pairs"
    assert launches(lambda: call(True, dy, wq, ws))[-1] == ("fp8_backward_pairs" if K > 2000 else "fp8_backward")
    dx = call(True, dy, wq, ws)
    want = float((dx.double() * step.double()).sum())
    a = dy.double().abs() @ wide_tiles(wq, ws).abs()
    mag = float(a.sum()) * 15 * 2 + float((a * step.double().abs()).sum())  # |x| <= 15
    assert abs(diff - want) <= (N * 2.0 ** -23 + (blocks(N) + 5) * 2.0 ** -24) * mag


# ------------------------------------------------------------------ the quantiser's form for large matrices

@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("rows,cols", [(2400, 1040), (2411, 1168), (40, 27664), (19000, 16)])
def test_quantize_equals_the_oracle(rows, cols, dtype, fp8, block):
    x = torch.randn(rows, cols, generator=gen(rows), device="cuda") * torch.exp2(
        torch.randint(-12, 12, (rows, blocks(cols)), generator=gen(cols), device="cuda").float()).repeat_interleave(128, 1)[:, :cols]
    x = x.to(dtype)
    x[rows // 2] = 0
    x[3, 5], x[rows - 1, cols - 1], x[rows // 3, 0] = float("inf"), float("nan"), 1e-40
    q, s = dw.dora_fp8_quantize(x, block=block, dtype=fp8)
    rq, rs = of.quantize(x.float().cpu().numpy().astype(np.float64), NAME[fp8], block == "tile")
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.float().cpu().numpy(), rq, equal_nan=True)
