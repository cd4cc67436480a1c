"""8-bit block quantisation and products on the GPU against the float64 oracle.

Quantisation is exact up to its one rounding, so codes and scales must equal
the oracle's. Products: with a_tk = |x_scale xq|, b_nk = |w_scale wq| the sum of
128 exact products in the tensor core's fp32 accumulator is off by at most
128 * 2^-23 of the block's sum of |products| (one unit in the last place per
addition, rounded or cut off), and folding nkb blocks with a rounded scale by at most
(nkb + 3) * 2^-24 of the whole; the result is then rounded once, by at most
half a step of the output type. Where the scales of a tile are powers of two,
the tensor core may apply them (exactly) and add all K products of a result in
the one accumulator: then the first bound is K * 2^-23 of the sum of |products|.
If those K roundings are independent, their sum is off by about
sqrt(K) * 2^-24 of the largest partial sum, so the whole matrix is also held to
sqrt(K) * 2^-22 of its norm (and the output's rounding).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from oracle import fp8 as of

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
NAME = {E4: "e4m3", E5: "e5m2"}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()
    yield
    assert dw.dora_device_status() == 0, "a kernel's bounded wait ran out"


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def matrix(rows, cols, dtype, seed=0, wide=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols))
    if wide:
        x *= np.exp2(rng.integers(-12, 12, (rows, -(-cols // 128)))).repeat(128, axis=1)[:, :cols]
    return torch.from_numpy(x).to(dtype).cuda()


def poisoned(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


# ------------------------------------------------------------------ quantisation

@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (127, 112), (128, 256), (129, 400), (300, 1040)])
def test_quantize_equals_the_oracle(rows, cols, dtype, fp8, block):
    x = matrix(rows, cols, dtype, seed=rows + cols)
    q, s = dw.dora_fp8_quantize(x, block=block, dtype=fp8)
    rq, rs = of.quantize(host(x), NAME[fp8], block == "tile")
    assert q.dtype == fp8 and tuple(s.shape) == rs.shape
    assert np.array_equal(host(s), rs)
    assert np.array_equal(host(q), rq)


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("fp8", [E4, E5])
def test_quantize_borders(fp8, block):
    """Zero blocks, subnormal and huge values, amax on and just over a power-of-two border, ties, infinities, NaN."""
    top = of.TOP[NAME[fp8]]
    vals = [0.0, 1e-45, 1e-38, 2.0 ** -126, 1e-30, top, np.nextafter(np.float32(top), np.float32(1e9)), top / 2,
            top * 2.0 ** -20, 1.0, 1.75, 1.7500001, 2.0, 3.0e38, np.inf, np.nan]
    x = np.zeros((len(vals) * 128, 128), np.float32)
    ties = np.arange(128) / 16.0 * (1 + 1 / 16)
    for i, v in enumerate(vals):
        x[i * 128] = ties * v / 8.5 if np.isfinite(v) else 1.0
        x[i * 128, 5] = v
        x[i * 128, 6] = -0.0
    d = torch.from_numpy(x).cuda()
    q, s = dw.dora_fp8_quantize(d, block=block, dtype=fp8)
    rq, rs = of.quantize(x, NAME[fp8], block == "tile")
    assert np.array_equal(host(s), rs, equal_nan=True)
    assert np.array_equal(host(q), rq, equal_nan=True)


def test_quantize_into_given_tensors_leaves_the_rest():
    x = matrix(37, 208, torch.bfloat16)
    qbuf = torch.full((40, 208), 3.0, device="cuda").to(E4)
    sbuf = poisoned(2 * 37 + 5)
    q, s = dw.dora_fp8_quantize(x, q=qbuf[:37], scale=sbuf[:74].view(2, 37))
    assert q.data_ptr() == qbuf.data_ptr()
    assert (qbuf[37:].float() == 3.0).all() and sbuf[74:].isnan().all() and not sbuf[:74].isnan().any()
    assert dw.dora_fp8_quantize(x[:0])[0].shape == (0, 208)


# ------------------------------------------------------------------ products

def weight(d_out, d_in, seed=1, pow2=False):
    rng = np.random.default_rng(seed)
    w = torch.from_numpy(rng.standard_normal((d_out, d_in)) * 100).cuda().to(E4)
    s = rng.uniform(0.5, 2.0, (-(-d_out // 128), -(-d_in // 128))) * np.exp2(rng.integers(-8, 4, (1, 1)))
    s = np.exp2(np.rint(np.log2(s))) if pow2 else s
    return w, torch.from_numpy(s.astype(np.float32)).cuda()


def check_product(out, a, b, K, what="", powers=False):
    """out against a @ b (float64), by the bounds of the module's first lines; powers: scales that are powers of two."""
    ref, mag = a @ b, np.abs(a) @ np.abs(b)
    sums = K if powers else 128
    tol = (sums * 2.0 ** -23 + (-(-K // 128) + 3) * 2.0 ** -24) * mag
    if not np.isnan(ref).any():
        far = np.linalg.norm(host(out) - ref) / max(np.linalg.norm(ref), 1e-300)
        assert far <= np.sqrt(K) * 2.0 ** -22 + HALF[out.dtype], (what, far)
    tol = tol + HALF[out.dtype] * (np.abs(ref) + tol)
    # An 8-bit NaN among the operands (the conversion of values beyond the type's range gives one) is a NaN in the result.
    nan = np.isnan(ref)
    assert np.array_equal(nan, np.isnan(host(out))), what
    err, tol, ref = np.where(nan, 0.0, np.abs(host(out) - ref)), np.where(nan, 1.0, tol), np.where(nan, 0.0, ref)
    worst = np.unravel_index(np.argmax(err / np.maximum(tol, 1e-300)), err.shape) if err.size else None
    assert np.all(err <= tol), (what, worst, err[worst], tol[worst], ref[worst])


SHAPES = [(1, 16, 16), (1, 128, 128), (1, 272, 1040), (2, 256, 144), (5, 1040, 272), (16, 384, 640), (17, 144, 4112),
          (33, 528, 128), (64, 2048, 256), (65, 128, 2064), (100, 400, 400), (127, 640, 384), (128, 128, 128),
          (129, 272, 272), (257, 528, 912), (300, 16, 656), (512, 1296, 336), (700, 640, 2048)]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T,d_out,d_in", SHAPES)
def test_products_of_given_codes(T, d_out, d_in, backward):
    """8-bit operands with arbitrary fp32 scales, float32 result; the buffers around the result stay."""
    K, N = (d_out, d_in) if backward else (d_in, d_out)
    fn = dw.dora_fp8_backward if backward else dw.dora_fp8_forward
    rng = np.random.default_rng(T)
    for fp8 in (E4, E5):
        xq = torch.from_numpy(rng.standard_normal((T, K)) * 50).cuda().to(fp8)
        xs = torch.from_numpy(rng.uniform(0.01, 3.0, (-(-K // 128), T)).astype(np.float32)).cuda()
        wq, ws = weight(d_out, d_in)
        buf = poisoned(T + 3, N)
        kw = {"dy_scale" if backward else "x_scale": xs, "dx" if backward else "y": buf[:T]}
        out = fn(xq, wq, ws, **kw)
        w = of.widen_tiles(host(wq), host(ws))
        check_product(out, of.widen_rows(host(xq), host(xs)), w if backward else w.T, K, (fp8, "codes"))
        assert buf[T:].isnan().all()


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d_out,d_in", [(1, 256, 512), (3, 1040, 272), (16, 400, 4624), (7, 16, 8208), (17, 144, 3600), (40, 272, 1168), (200, 528, 400), (513, 656, 784)])
def test_products_of_wide_operands(T, d_out, d_in, dtype, backward):
    """bf16 and float32 operands, quantised in the call: equal to the product of the oracle's codes."""
    K = d_out if backward else d_in
    fn = dw.dora_fp8_backward if backward else dw.dora_fp8_forward
    x = matrix(T, K, dtype, seed=T)
    wq, ws = dw.dora_fp8_quantize(matrix(d_out, d_in, torch.bfloat16, seed=2, wide=False), block="tile")
    w = of.widen_tiles(host(wq), host(ws))
    for fp8 in (E4, E5):
        out = fn(x, wq, ws, fp8_dtype=fp8)
        assert out.dtype == dtype
        q, s = of.quantize(host(x), NAME[fp8], False)
        check_product(out, of.widen_rows(q, s), w if backward else w.T, K, fp8, powers=True)
        # the two-call form gives the same bits
        xq, xs = dw.dora_fp8_quantize(x, dtype=fp8)
        two = fn(xq, wq, ws, out_dtype=dtype, **{"dy_scale" if backward else "x_scale": xs})
        assert torch.equal(out, two)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("T,d_out,d_in", [(129, 256, 128), (256, 272, 1168), (300, 528, 400), (517, 1040, 272), (140, 144, 27648),
                                           (17, 400, 528), (70, 1040, 2064), (128, 272, 272), (16, 144, 27648)])
def test_scales_that_are_powers_of_two_and_others(T, d_out, d_in, backward):
    """The tensor cores apply the scales of the first call; one scale of the weight, or of the operand, in the later ones
    is no power of two, zero, negative or subnormal, and those are applied in fp32."""
    K = d_out if backward else d_in
    fn = dw.dora_fp8_backward if backward else dw.dora_fp8_forward
    rng = np.random.default_rng(T)
    xq = torch.from_numpy(rng.standard_normal((T, K)) * 50).cuda().to(E4)
    wq = torch.from_numpy(rng.standard_normal((d_out, d_in)) * 50).cuda().to(E4)
    xs0 = torch.from_numpy(np.exp2(rng.integers(-20, 20, (-(-K // 128), T))).astype(np.float32)).cuda()
    ws0 = torch.from_numpy(np.exp2(rng.integers(-9, 9, (-(-d_out // 128), -(-d_in // 128)))).astype(np.float32)).cuda()
    key = "dy_scale" if backward else "x_scale"
    for what, at, v in (("powers", None, 1), ("weight", "w", 1.5), ("operand", "x", 0.7), ("zero", "w", 0.0), ("negative", "w", -2.0),
                        ("subnormal", "x", 1e-40)):
        xs, ws = xs0.clone(), ws0.clone()
        if at == "w":
            ws.view(-1)[-1] = v
        elif at == "x":
            xs.view(-1)[xs.numel() // 2] = v
        out = fn(xq, wq, ws, out_dtype=torch.float32, **{key: xs})
        w = of.widen_tiles(host(wq), host(ws))
        check_product(out, of.widen_rows(host(xq), host(xs)), w if backward else w.T, K, what, powers=True)  # those of other tiles stay


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T", [1, 9, 24, 100, 140, 300])
def test_non_finite_rows_stay_in_their_rows(T, pow2):
    x = matrix(T, 384, torch.bfloat16, wide=False)
    wq, ws = weight(272, 384, pow2=pow2)
    clean = dw.dora_fp8_forward(x, wq, ws)
    x[0, 200] = float("inf")
    if T > 5:
        x[4, 7] = float("nan")
    out = dw.dora_fp8_forward(x, wq, ws)
    bad = [0] + ([4] if T > 5 else [])
    keep = [i for i in range(T) if i not in bad]
    assert not torch.isfinite(out[bad]).any()
    assert torch.equal(out[keep], clean[keep])


def test_zero_rows_and_zero_scales():
    x = matrix(200, 256, torch.bfloat16, wide=False)
    x[13] = 0
    wq, ws = weight(256, 256)
    ws[1] = 0
    y = dw.dora_fp8_forward(x, wq, ws)
    assert (y[13] == 0).all() and (y[:, 128:] == 0).all() and (y[:13, :128] != 0).any()


def test_no_tokens():
    wq, ws = weight(256, 128)
    assert dw.dora_fp8_forward(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), wq, ws).shape == (0, 256)
    assert dw.dora_fp8_backward(torch.empty(0, 256, dtype=torch.float32, device="cuda"), wq, ws).shape == (0, 128)


@pytest.mark.parametrize("T", [1, 48, 600])
def test_gradient_by_differences(T):
    """dx = dy W is the derivative of sum(dy y) along any direction (exact codes, so no rounding of x intervenes)."""
    rng = np.random.default_rng(T)
    wq, ws = weight(272, 400, pow2=True)
    x0 = torch.from_numpy(rng.integers(-8, 9, (T, 400)).astype(np.float32)).cuda()
    dirn = torch.from_numpy(rng.integers(-7, 8, (T, 400)).astype(np.float32)).cuda()
    dy = torch.from_numpy(rng.integers(-8, 9, (T, 272)).astype(np.float32)).cuda()
    f = lambda x: float((host(dw.dora_fp8_forward(x, wq, ws)) * host(dy)).sum())
    diff = f(x0 + dirn) - f(x0)
    dx = dw.dora_fp8_backward(dy, wq, ws)
    want = float((host(dx) * host(dirn)).sum())
    w = of.widen_tiles(host(wq), host(ws))
    # three results, each an fp32 sum within the products' bound of its sum of magnitudes (|x| <= 15 here)
    mag = float((np.abs(host(dy)) @ np.abs(w)).sum()) * 15 * 2 + float((np.abs(host(dy)) @ np.abs(w) * np.abs(host(dirn))).sum())
    sums = 400  # products added in one accumulator at most (d_in = 400, d_out = 272)
    assert abs(diff - want) <= (sums * 2.0 ** -23 + 10 * 2.0 ** -24) * mag


def test_stream_and_graph():
    """On a stream of its own, and captured and replayed with new inputs, the bits are the eager call's."""
    x = [matrix(70, 528, torch.bfloat16, seed=i) for i in range(3)]
    dy = [matrix(70, 400, torch.float32, seed=10 + i) for i in range(3)]
    wq, ws = weight(400, 528)
    ref = [(dw.dora_fp8_forward(a, wq, ws), dw.dora_fp8_backward(b, wq, ws)) for a, b in zip(x, dy)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = [(dw.dora_fp8_forward(a, wq, ws, stream=st), dw.dora_fp8_backward(b, wq, ws, stream=st)) for a, b in zip(x, dy)]
    st.synchronize()
    for r, g in zip(ref, got):
        assert torch.equal(r[0], g[0]) and torch.equal(r[1], g[1])
    sx, sdy = x[0].clone(), dy[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = dw.dora_fp8_forward(sx, wq, ws), dw.dora_fp8_backward(sdy, wq, ws)
    for i in (1, 2, 1):
        sx.copy_(x[i])
        sdy.copy_(dy[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref[i][0]) and torch.equal(dx, ref[i][1])


@pytest.mark.parametrize("T", [1, 24, 200])
def test_two_calls_at_once(T):
    """Calls on two streams share nothing."""
    wq, ws = weight(1040, 1168)
    xs = [matrix(T, 1168, torch.bfloat16, seed=i) for i in range(2)]
    ref = [dw.dora_fp8_forward(x, wq, ws) for x in xs]
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream() for _ in xs]
    outs = [[] for _ in xs]
    for _ in range(20):
        for o, x, st in zip(outs, xs, sts):
            o.append(dw.dora_fp8_forward(x, wq, ws, stream=st))
    torch.cuda.synchronize()
    for r, o in zip(ref, outs):
        assert all(torch.equal(r.view(torch.int16), v.view(torch.int16)) for v in o)  # bits: a NaN weight gives NaN


def test_refusals_on_the_device():
    wq, ws = weight(256, 128)
    x = matrix(4, 128, torch.bfloat16)
    with pytest.raises(dw.DoraError, match="EWORKSPACE"):
        dw.dora_fp8_forward(matrix(20, 128, torch.bfloat16), wq, ws, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="ws is on cpu"):
        dw.dora_fp8_forward(matrix(20, 128, torch.bfloat16), wq, ws, ws=torch.empty(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        dw.dora_fp8_forward(matrix(4, 256, torch.bfloat16)[:, :128], wq, ws)
    buf = torch.zeros(4 * 128 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dw.DoraError, match="aligned"):
        dw.dora_fp8_forward(buf[1:1 + 512].view(4, 128), wq, ws)
    other = torch.cuda.Stream()
    assert torch.equal(dw.dora_fp8_forward(x, wq, ws), dw.dora_fp8_forward(x, wq, ws, stream=other))
