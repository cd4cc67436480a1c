"""Workspaces that the caller gives to the operators around the layer, checked without a GPU."""
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from dora_weight_decomposed_b200 import build as dbuild


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dbuild.build()


def test_a_workspace_on_another_device_is_refused():
    other = torch.empty(1 << 16, dtype=torch.uint8, device="meta")
    with pytest.raises(ValueError, match="ws is on meta, expected cpu"):
        dw.dora_grad_norm([torch.zeros(4)], ws=other)
    wq, ws = torch.zeros(256, 144, dtype=torch.float8_e4m3fn), torch.ones(2, 2)
    for call in (lambda: dw.dora_fp8_forward(torch.zeros(30, 144), wq, ws, ws=other),
                 lambda: dw.dora_fp8_backward(torch.zeros(30, 256), wq, ws, ws=other)):
        with pytest.raises(ValueError, match="ws is on meta, expected cpu"):
            call()
