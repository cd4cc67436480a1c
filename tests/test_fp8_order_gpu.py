"""The 8-bit products give the same bits whichever call of a process comes first: what a call asks the device (how many
clusters it holds at once, from which the splits of K follow) has one answer."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import hashlib, sys
sys.path.insert(0, {root!r})
import torch
import dora_weight_decomposed_b200 as dw

def bits(T, tiles, backward, given):
    g = torch.Generator(device="cuda").manual_seed(tiles)
    K, N = 8192, 128 * tiles
    shape = (K, N) if backward else (N, K)
    w = torch.randn(*shape, generator=g, device="cuda").clamp(-4, 4).to(torch.float8_e4m3fn)
    s = torch.ones(shape[0] // 128, shape[1] // 128, device="cuda")
    x = torch.randn(T, K, generator=g, device="cuda")
    fn = dw.dora_fp8_backward if backward else dw.dora_fp8_forward
    kw = dict(out_dtype=torch.float32)
    if given:
        x, kw["dy_scale" if backward else "x_scale"] = dw.dora_fp8_quantize(x)
    return hashlib.sha1(fn(x, w, s, **kw).cpu().numpy().tobytes()).hexdigest()

for arg in sys.argv[1:]:  # the calls in front
    T, given = arg.split(",")
    for backward in (False, True):
        bits(int(T), 1, backward, given == "codes")
for tiles in (32, 42, 46, 52, 60, 70, 88, 140):  # around what a B200 holds of clusters of 8 to 2 CTAs
    for T, given in ((100, False), (16, False), (16, True), (40, False)):
        for backward in (False, True):
            print(tiles, T, given, backward, bits(T, tiles, backward, given))
assert dw.dora_device_status() == 0
"""


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()


def test_the_first_call_does_not_matter():
    out = [subprocess.run([sys.executable, "-c", CODE.format(root=ROOT), *first], capture_output=True, text=True, timeout=300)
           for first in (["100,wide", "16,codes", "300,wide"], ["300,wide", "16,wide", "100,wide"], ["1,wide"])]
    for o in out:
        assert o.returncode == 0, o.stderr
    lines = [o.stdout.splitlines() for o in out]
    assert len(lines[0]) == 64
    for other in lines[1:]:
        assert [a for a, b in zip(lines[0], other) if a != b] == []
