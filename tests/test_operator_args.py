"""Refusals of the 8-bit products, the quantiser, the gradient norm and the AdamW step, without a GPU:
the binding's checks of types, shapes and bindings, and the C ABI's checks, which all
come before anything is launched. Every C call below that passes placeholder pointers
fails one of them. Valid arguments on the CPU get as far as the device check.
"""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from dora_weight_decomposed_b200 import adamw as da
from dora_weight_decomposed_b200 import build as dbuild
from dora_weight_decomposed_b200 import fp8 as df

CUDA_ONLY = "tensors must be on a CUDA device"
BF, F32, E4, E5 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2
FAKE = 4096


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dw.load_library()


def _weight(d_out=256, d_in=144):
    return torch.zeros(d_out, d_in, dtype=E4), torch.ones(-(-d_out // 128), -(-d_in // 128))


def test_valid_arguments_reach_the_device_check():
    wq, ws = _weight()
    for call in (lambda: dw.dora_fp8_quantize(torch.zeros(5, 144, dtype=BF)),
                 lambda: dw.dora_fp8_quantize(torch.zeros(5, 144), block="tile", dtype=E5),
                 lambda: dw.dora_fp8_forward(torch.zeros(3, 144, dtype=BF), wq, ws),
                 lambda: dw.dora_fp8_forward(torch.zeros(3, 144, dtype=E4), wq, ws, x_scale=torch.ones(2, 3)),
                 lambda: dw.dora_fp8_backward(torch.zeros(3, 256), wq, ws, fp8_dtype=E5, out_dtype=BF),
                 lambda: dw.dora_grad_norm([torch.zeros(4)]),
                 lambda: dw.DoraAdamW([torch.zeros(4)], [torch.zeros(4)], lr=0.1)):
        with pytest.raises(ValueError, match=CUDA_ONLY):
            call()


@pytest.mark.parametrize("kw,error,match", [
    (dict(x=torch.zeros(3, 128, dtype=BF)), ValueError, "x has shape"),
    (dict(x=torch.zeros(3, 144, dtype=torch.float16)), TypeError, "x is"),
    (dict(x=torch.zeros(144, dtype=BF)), ValueError, "matrices"),
    (dict(x=torch.zeros(3, 144, dtype=E4)), ValueError, "needs x_scale"),
    (dict(x_scale=torch.ones(2, 3)), ValueError, "quantised in the call"),
    (dict(x=torch.zeros(3, 144, dtype=E5), x_scale=torch.ones(3, 2)), ValueError, "x_scale has shape"),
    (dict(wq=torch.zeros(256, 144, dtype=E5)), TypeError, "wq is"),
    (dict(w_scale=torch.ones(2, 1)), ValueError, "w_scale has shape"),
    (dict(w_scale=torch.ones(2, 2, dtype=torch.float64)), TypeError, "w_scale is"),
    (dict(y=torch.zeros(3, 255, dtype=BF)), ValueError, "y has shape"),
    (dict(out_dtype=F32, y=torch.zeros(3, 256, dtype=BF)), TypeError, "y is"),
    (dict(out_dtype=E4), TypeError, "out_dtype is"),
    (dict(fp8_dtype=BF), TypeError, "fp8_dtype is")])
def test_forward_refusals(kw, error, match):
    wq, ws = _weight()
    a = dict(dict(x=torch.zeros(3, 144, dtype=BF), wq=wq, w_scale=ws), **kw)
    with pytest.raises(error, match=match):
        dw.dora_fp8_forward(a.pop("x"), a.pop("wq"), a.pop("w_scale"), **a)


def test_backward_and_quantize_refusals():
    wq, ws = _weight()
    with pytest.raises(ValueError, match="dy has shape"):
        dw.dora_fp8_backward(torch.zeros(3, 144, dtype=BF), wq, ws)
    with pytest.raises(ValueError, match="needs dy_scale"):
        dw.dora_fp8_backward(torch.zeros(3, 256, dtype=E5), wq, ws)
    with pytest.raises(ValueError, match="block is"):
        dw.dora_fp8_quantize(torch.zeros(3, 144), block="column")
    with pytest.raises(TypeError, match="dtype is"):
        dw.dora_fp8_quantize(torch.zeros(3, 144), dtype=BF)
    with pytest.raises(ValueError, match="dimensions"):
        dw.dora_fp8_quantize(torch.zeros(144))
    with pytest.raises(ValueError, match="scale has shape"):
        dw.dora_fp8_quantize(torch.zeros(3, 144), scale=torch.ones(3, 2))


def test_adamw_refusals():
    z = torch.zeros
    with pytest.raises(ValueError, match="0 parameters"):
        dw.DoraAdamW([], [], lr=0.1)
    with pytest.raises(ValueError, match="1 parameters and 2"):
        dw.DoraAdamW([z(4)], [z(4), z(4)], lr=0.1)
    with pytest.raises(ValueError, match="state_bits"):
        dw.DoraAdamW([z(4)], [z(4)], lr=0.1, state_bits=16)
    with pytest.raises(ValueError, match="weight decays"):
        dw.DoraAdamW([z(4)], [z(4)], lr=0.1, weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError, match="gradient 0 has shape"):
        dw.DoraAdamW([z(4)], [z(5)], lr=0.1)
    with pytest.raises(TypeError, match="parameter 0 is"):
        dw.DoraAdamW([z(4, dtype=torch.float64)], [z(4)], lr=0.1)
    with pytest.raises(ValueError, match="empty"):
        dw.dora_grad_norm([])


# ------------------------------------------------------------------ C ABI

def _desc(d_out=256, d_in=144, i=0, f=2, o=0):
    return df.Fp8Desc(d_out, d_in, i, f, o)


@pytest.mark.parametrize("bad", [dict(d_out=0), dict(d_out=250), dict(d_in=8), dict(i=7), dict(f=0), dict(o=2),
                                 dict(d_in=1 << 40)])
def test_fp8_descriptors(lib, bad):
    d = _desc(**bad)
    assert lib.dora_fp8_workspace_size(ctypes.byref(d), 4, 0) == 0
    for fn in (lib.dora_fp8_forward, lib.dora_fp8_backward):
        assert fn(ctypes.byref(d), 4, FAKE, None, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == 1
        assert dw.dora_last_error()


def test_fp8_pointers_and_workspace(lib):
    d = _desc()
    assert lib.dora_fp8_workspace_size(ctypes.byref(d), 16, 0) == 0  # few tokens are quantised where they are used
    need = lib.dora_fp8_workspace_size(ctypes.byref(d), 50, 0)
    assert need >= 50 * 144 + 2 * 50 * 4 and need % 256 == 0
    assert lib.dora_fp8_workspace_size(ctypes.byref(d), 50, 1) >= 50 * 256 + 2 * 50 * 4
    assert lib.dora_fp8_workspace_size(ctypes.byref(d), 5, 2) == 0
    f = lambda *a: lib.dora_fp8_forward(ctypes.byref(d), *a)
    assert f(5, None, None, FAKE, FAKE, FAKE, FAKE, need, None) == 1 and "x is NULL" in dw.dora_last_error()
    assert f(5, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, need, None) == 1 and "x_scale" in dw.dora_last_error()
    assert f(5, FAKE + 8, None, FAKE, FAKE, FAKE, FAKE, need, None) == 1 and "aligned" in dw.dora_last_error()
    assert f(5, FAKE, None, FAKE, None, FAKE, FAKE, need, None) == 1 and "w_scale" in dw.dora_last_error()
    assert f(50, FAKE, None, FAKE, FAKE, FAKE, None, 0, None) == 3
    assert f(50, FAKE, None, FAKE, FAKE, FAKE, FAKE, need - 1, None) == 3
    assert f(50, FAKE, None, FAKE, FAKE, FAKE, FAKE + 16, need, None) == 1
    assert f(-1, FAKE, None, FAKE, FAKE, FAKE, FAKE, need, None) == 1
    q = lambda *a: lib.dora_fp8_quantize(*a)
    assert q(4, 100, 0, 2, 0, FAKE, FAKE, FAKE, None) == 1 and "16" in dw.dora_last_error()
    assert q(4, 128, 2, 2, 0, FAKE, FAKE, FAKE, None) == 1
    assert q(4, 128, 0, 1, 0, FAKE, FAKE, FAKE, None) == 1
    assert q(4, 128, 0, 2, 5, FAKE, FAKE, FAKE, None) == 1
    assert q(-1, 128, 0, 2, 0, FAKE, FAKE, FAKE, None) == 1
    assert q(4, 128, 0, 2, 0, FAKE, None, FAKE, None) == 1 and "q is NULL" in dw.dora_last_error()


def _row(**kw):
    a = dict(param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, scale_avg=FAKE, scale_sq=FAKE, master=None, numel=10,
             index0=0, weight_decay=0.0, param_dtype=0, grad_dtype=0)
    a.update(kw)
    return da.AdamwTensor(**a)


@pytest.mark.parametrize("bad,word", [
    (dict(param=None), "param"), (dict(grad=FAKE + 1), "grad"), (dict(exp_avg=FAKE + 8), "exp_avg"),
    (dict(exp_avg_sq=None), "exp_avg_sq"), (dict(scale_avg=None), "scale_avg"), (dict(master=FAKE + 4), "master"),
    (dict(numel=-1), "numel"), (dict(index0=4), "index0"), (dict(weight_decay=float("inf")), "weight_decay"),
    (dict(param_dtype=2), "dtype"), (dict(grad_dtype=9), "dtype"), (dict(param=FAKE + 2, param_dtype=1), "param")])
def test_adamw_tensors(lib, bad, word):
    d = da.AdamwDesc(0.9, 0.999, 1e-8, 8, 0)
    t = (da.AdamwTensor * 2)(_row(numel=0), _row(**bad))
    assert lib.dora_adamw(ctypes.byref(d), t, 2, FAKE, None, None) == 1
    assert "tensor 1" in dw.dora_last_error() and word in dw.dora_last_error()


@pytest.mark.parametrize("d", [da.AdamwDesc(1.0, 0.999, 1e-8, 8, 0), da.AdamwDesc(0.9, -0.1, 1e-8, 8, 0),
                               da.AdamwDesc(0.9, 0.999, -1.0, 8, 0), da.AdamwDesc(0.9, 0.999, 1e-8, 16, 0),
                               da.AdamwDesc(float("nan"), 0.999, 1e-8, 32, 0)])
def test_adamw_descriptors(lib, d):
    t = (da.AdamwTensor * 1)(_row())
    assert lib.dora_adamw(ctypes.byref(d), t, 1, FAKE, None, None) == 1


def test_adamw_and_norm_pointers(lib):
    d = da.AdamwDesc(0.9, 0.999, 1e-8, 8, 0)
    t = (da.AdamwTensor * 1)(_row())
    assert lib.dora_adamw(ctypes.byref(d), t, 1, None, None, None) == 1 and "control" in dw.dora_last_error()
    assert lib.dora_adamw(ctypes.byref(d), None, 1, FAKE, None, None) == 1
    assert lib.dora_adamw(None, t, 1, FAKE, None, None) == 1
    g = (da.GradEntry * 1)(da.GradEntry(FAKE, 10, 0))
    need = lib.dora_grad_norm_workspace_size(1)
    assert need > 0 and lib.dora_grad_norm_workspace_size(-1) == 0
    assert lib.dora_grad_norm(g, 1, 1.0, FAKE, FAKE, FAKE, need - 1, None) == 3
    assert lib.dora_grad_norm(g, 1, 0.0, FAKE, FAKE, FAKE, need, None) == 1
    assert lib.dora_grad_norm(g, 1, float("nan"), FAKE, FAKE, FAKE, need, None) == 1
    assert lib.dora_grad_norm(g, 1, 1.0, None, FAKE, FAKE, need, None) == 1
    c = lambda *a: lib.dora_adamw_clipped(ctypes.byref(d), t, 1, FAKE, *a, None)
    assert c(1.0, None, FAKE, need) == 1 and "norm" in dw.dora_last_error()
    assert c(-1.0, FAKE, FAKE, need) == 1 and "max_norm" in dw.dora_last_error()
    assert c(1.0, FAKE, FAKE, need - 1) == 3
    assert c(1.0, FAKE, None, need) == 3
    bad = (da.GradEntry * 1)(da.GradEntry(FAKE + 1, 10, 0))
    assert lib.dora_grad_norm(bad, 1, 1.0, FAKE, FAKE, FAKE, need, None) == 1
