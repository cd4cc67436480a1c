"""The 8-bit calls and the AdamW step called in ways of their own: first thing in a process inside a graph capture, from
two host threads, on tensors that a padded batch leaves, over long matrices, and with the kernel profiler on.
"""
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()
    yield
    assert dw.dora_device_status() == 0, "a kernel's bounded wait ran out"


def weight(d_out, d_in, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return dw.dora_fp8_quantize(torch.randn(d_out, d_in, generator=g, device="cuda") * 0.05, block="tile")


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import dora_weight_decomposed_b200 as dw
g = torch.Generator(device="cuda").manual_seed(1)
x = [torch.randn(T, 528, generator=g, device="cuda").bfloat16() for T in (1, 40, 300)]
W = torch.randn(400, 528, generator=g, device="cuda") * 0.05
p, dp = torch.randn(5000, generator=g, device="cuda"), torch.randn(5000, generator=g, device="cuda")
p0 = p.clone()
opt = dw.DoraAdamW([p], [dp], lr=1e-2, state_bits=8)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    wq, ws = dw.dora_fp8_quantize(W, block="tile")
    y = [dw.dora_fp8_forward(v, wq, ws) for v in x]
    dx = [dw.dora_fp8_backward(v, wq, ws) for v in y]
    norm = opt.step(max_norm=1.0)
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
eq, es = dw.dora_fp8_quantize(W, block="tile")
assert torch.equal(eq.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(es, ws)
for v, a, b in zip(x, y, dx):
    assert torch.equal(dw.dora_fp8_forward(v, eq, es), a)
    assert torch.equal(dw.dora_fp8_backward(a, eq, es), b)
assert int(opt.state_dict()["step"]) == 2 and (p != p0).all()
q = p0.clone()
eager = dw.DoraAdamW([q], [dp], lr=1e-2, state_bits=8)
for _ in range(2):
    eager.step(max_norm=1.0)
assert torch.equal(p, q)
assert dw.dora_device_status() == 0
print("first call captured")
"""


def test_first_call_of_a_process_is_captured():
    out = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "first call captured" in out.stdout, out.stdout + out.stderr


def test_two_host_threads():
    wq, ws = weight(1040, 784)
    xs = [torch.randn(T, 784, device="cuda").to(BF) for T in (3, 90, 260)]
    ref = [dw.dora_fp8_forward(x, wq, ws) for x in xs]
    p0, g = torch.randn(10000, device="cuda"), torch.randn(10000, device="cuda")
    q = p0.clone()
    opt = dw.DoraAdamW([q], [g], lr=1e-2, state_bits=8)
    for _ in range(30):
        opt.step(max_norm=1.0)
    torch.cuda.synchronize()
    bad = []

    def work(seed):
        st = torch.cuda.Stream()
        p = p0.clone()
        mine = dw.DoraAdamW([p], [g], lr=1e-2, state_bits=8)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for i in range(30):
                k = (i + seed) % 3
                if not torch.equal(dw.dora_fp8_forward(xs[k], wq, ws), ref[k]):
                    bad.append((seed, i))
                mine.step(max_norm=1.0)
        st.synchronize()
        if not torch.equal(p, q):
            bad.append((seed, "step"))

    threads = [threading.Thread(target=work, args=(s,)) for s in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("T", [1, 33, 200, 300])
def test_a_padded_batch(T):
    """The first T rows of longer buffers: rows behind them are neither read nor written."""
    wq, ws = weight(528, 400)
    x = torch.full((T + 9, 400), float("nan"), dtype=BF, device="cuda")
    x[:T] = torch.randn(T, 400, device="cuda")
    y = torch.full((T + 9, 528), 7.0, dtype=BF, device="cuda")
    dw.dora_fp8_forward(x[:T], wq, ws, y=y[:T])
    assert torch.isfinite(y[:T]).all() and (y[T:] == 7).all()
    assert torch.equal(y[:T], dw.dora_fp8_forward(x[:T].clone(), wq, ws))
    dx = torch.full((T + 9, 400), 7.0, device="cuda")
    dw.dora_fp8_backward(y[:T], wq, ws, dx=dx[:T], out_dtype=torch.float32)
    assert torch.isfinite(dx[:T]).all() and (dx[T:] == 7).all()


def test_offsets_beyond_32_bits():
    """A quantised matrix and a result of more than 2^31 elements: the last rows are those of a short call. A short call
    may split its sums another way. Either result is off by K * 2^-23 of the sum of its K products' magnitudes and, to
    bf16, 2^-8 of itself, with (K / 128 + 3) * 2^-24 more where blocks are added in fp32; two differ by twice that."""
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    T = 270_000
    x = torch.zeros(T, 8192, dtype=BF, device="cuda")  # 2.2e9 elements
    x[-300:] = torch.randn(300, 8192, device="cuda")
    q, s = dw.dora_fp8_quantize(x)
    q0, s0 = dw.dora_fp8_quantize(x[-300:].clone())
    assert torch.equal(q[-300:].view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s[:, -300:], s0)
    wq, ws = weight(256, 8192)
    y = dw.dora_fp8_forward(q, wq, ws, x_scale=s)
    short = dw.dora_fp8_forward(q0, wq, ws, x_scale=s0).double()
    wide = lambda q, s: q.double() * s.double().T.repeat_interleave(128, 1)
    w = wq.double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    mag = wide(q0, s0).abs() @ w.abs().T
    tol = 2 * (8192 * 2.0 ** -23 + 67 * 2.0 ** -24) * mag
    tol = tol + 2.0 ** -8 * (y[-300:].double().abs() + short.abs())
    assert ((y[-300:].double() - short).abs() <= tol).all() and (y[:1000] == 0).all()
    del q, s, y
    small = torch.randn(300, 256, device="cuda").to(BF)
    dy = torch.zeros(T, 256, dtype=BF, device="cuda")
    dy[-300:] = small
    dx = dw.dora_fp8_backward(dy, wq, ws, dx=x)  # 2.2e9 results, over x
    short = dw.dora_fp8_backward(small, wq, ws).double()
    mag = wide(*dw.dora_fp8_quantize(small)).abs() @ w.abs()
    tol = 2 * (256 * 2.0 ** -23 + 5 * 2.0 ** -24) * mag + 2.0 ** -8 * (dx[-300:].double().abs() + short.abs())
    assert ((dx[-300:].double() - short).abs() <= tol).all() and (dx[:1000] == 0).all()


def test_profiler_names_the_kernels():
    wq, ws = weight(256, 256)
    p, g = torch.randn(300, device="cuda"), torch.randn(300, device="cuda")
    opt = dw.DoraAdamW([p], [g], lr=0.1)
    dw.dora_profile_start(64)
    dw.dora_fp8_forward(torch.randn(200, 256, device="cuda"), wq, ws)
    dw.dora_fp8_backward(torch.randn(2, 256, device="cuda"), wq, ws)
    opt.step(max_norm=1.0)
    torch.cuda.synchronize()
    names = [n for n, _ in dw.dora_profile_read()]
    dw.dora_profile_stop()
    assert names == ["fp8_quantize_rows", "fp8_forward", "fp8_backward", "grad_norm_partial", "adamw32"]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("numel", [3_000, 400_000, 9_000_000])
def test_steps_in_a_row_and_fresh_parameters(numel, bits):
    """Clipped steps right behind one another, and behind kernels that have just written the parameters and gradients,
    give the bits of steps with a wait before each: an update reads nothing ahead of the work before it."""
    gen = torch.Generator(device="cuda").manual_seed(numel + bits)
    p0 = torch.randn(numel, generator=gen, device="cuda").to(BF)
    gs = [torch.randn(numel, generator=gen, device="cuda").to(BF) for _ in range(3)]

    def run(wait):
        p, g = p0.clone(), gs[0].clone()
        opt = dw.DoraAdamW([p], [g], lr=0.01, state_bits=bits, master=False)
        norms = []
        torch.cuda.synchronize()
        for i in range(12):
            g.copy_(gs[i % 3])
            if i % 4 == 3:
                p.mul_(0.5)
            if wait:
                torch.cuda.synchronize()
            norms.append(opt.step(max_norm=1.0))
            if i % 5 == 4:
                norms.append(opt.step(max_norm=2.0))
        state = opt.state_dict()
        return [p, torch.stack(norms)] + [v.view(torch.uint8) for v in (state["avg"], state["sq"])]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
