"""The calls in the order a fine-tune makes them: an adapted layer behind a frozen 8-bit layer is
stepped with AdamW, then merged, quantised and served in 8 bits. Each stage is checked
against the oracle on the values that the stage before it left on the device.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dora_testlib as tl
import dora_weight_decomposed_b200 as dw
import oracle
from dora_inputs import make_inputs, workload
from oracle import adamw as oa
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


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("bits,master", [(32, True), (8, False), (8, True)])
@pytest.mark.parametrize("T", [1, 150])
def test_train_merge_and_serve(bits, master, T):
    wl = workload("c3", d_out=320, d_in=448, r=136, T=T)
    inp = make_inputs(wl)
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.bfloat16).contiguous()
    W0, A, B, dy = bf(inp["W0"]), bf(inp["A"]), bf(inp["B"]), bf(inp["dy"])
    m = torch.from_numpy(inp["m"]).cuda()
    rng = np.random.default_rng(4)
    x0 = bf(rng.standard_normal((T, 272)))
    fq, fs = dw.dora_fp8_quantize(bf(rng.standard_normal((448, 272)) * 0.06), block="tile")  # the frozen layer before it
    grads = [torch.zeros_like(t) for t in (A, B, m)]
    opt = dw.DoraAdamW([A, B, m], grads, lr=1e-3, state_bits=bits, master=master, weight_decay=[0.01, 0.01, 0.0])
    frozen = of.widen_tiles(host(fq), host(fs))
    for t in (1, 2):
        x = dw.dora_fp8_forward(x0, fq, fs)
        q, s = of.quantize(host(x0), "e4m3", False)
        ref = of.widen_rows(q, s) @ frozen.T
        assert np.linalg.norm(host(x) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
        C, g, gm1 = dw.dora_norm(W0, A, B, m, wl.s)
        y, su, pre = dw.dora_forward(x, W0, A, B, gm1, wl.s)
        _, _, _, dx = dw.dora_backward(dy, x, W0, A, B, C, g, su, pre, wl.s, dm=grads[2], dA=grads[0], dB=grads[1])
        rg = oracle.backward(host(dy), host(x), host(W0), host(A), host(B), host(m), wl.s)
        for name, got in (("dA", grads[0]), ("dB", grads[1]), ("dm", grads[2])):
            assert np.linalg.norm(host(got) - rg[name]) <= 2e-2 * np.linalg.norm(rg[name]), name
        dx0 = dw.dora_fp8_backward(dx, fq, fs)
        q, s = of.quantize(host(dx), "e4m3", False)
        ref = of.widen_rows(q, s) @ frozen
        assert np.linalg.norm(host(dx0) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
        before = [p.clone() for p in (A, B, m)]
        norm = opt.step(max_norm=1.0)
        rn, _ = oa.grad_norm([host(v) for v in grads], 1.0)
        assert abs(float(norm) - rn) <= 1e-6 * rn
        if t == 1:  # from zero moments every element moves by lr against its gradient's sign
            for p, b, gr in zip((A, B, m), before, grads):
                step = host(p) - host(b) * (1 - 1e-3 * (0.01 if p is not m else 0.0))
                half = 2.0 ** -8 if p.dtype == torch.bfloat16 else 2.0 ** -23
                live = np.abs(host(gr)) > 1e-4 * np.abs(host(gr)).max()
                # v = (1 - b2) g^2: the step is lr g' / (|g'| + eps), g' the clipped gradient
                gc = np.abs(host(gr)) / max(1.0, rn)
                tol = half * np.abs(host(p)) + 1e-3 * (1e-5 + 1e-8 / gc)
                assert np.all(np.abs(step + 1e-3 * np.sign(host(gr)))[live] <= tol[live])
    C, g, gm1 = dw.dora_norm(W0, A, B, m, wl.s)
    merged = dw.dora_merge(W0, A, B, g, wl.s)
    wq, ws = dw.dora_fp8_quantize(merged, block="tile")
    rq, rs = of.quantize(host(merged), "e4m3", True)
    assert np.array_equal(host(wq), rq) and np.array_equal(host(ws), rs)
    x = bf(rng.standard_normal((T, 448)))
    y = dw.dora_fp8_forward(x, wq, ws)
    q, s = of.quantize(host(x), "e4m3", False)
    ref = of.widen_rows(q, s) @ of.widen_tiles(rq, rs).T
    assert np.linalg.norm(host(y) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
