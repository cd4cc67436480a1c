"""Linear layers held in 8-bit floats: block quantisation and the two products.

    wq, w_scale = dora_fp8_quantize(W, block="tile")      # a merged or frozen weight, once
    y  = dora_fp8_forward(x, wq, w_scale)                  # x W^T; x is quantised in the call
    dx = dora_fp8_backward(dy, wq, w_scale)                # dy W: W is frozen and gets no gradient

    xq, x_scale = dora_fp8_quantize(x, block="row")        # one quantisation for several layers
    y = dora_fp8_forward(xq, wq, w_scale, x_scale=x_scale)

One fp32 scale per 128 x 128 block of W and per 1 x 128 block of x or dy; see
include/dora.h for the formulas.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import _check, _ptr, _shape, _stream_ptr, _torch, load_library

DORA_E4M3, DORA_E5M2 = 2, 3
DORA_FP8_OP_FORWARD, DORA_FP8_OP_BACKWARD = 0, 1
_BLOCKS = {"row": 0, "tile": 1}


class Fp8Desc(ctypes.Structure):
    _fields_ = [("d_out", ctypes.c_int64), ("d_in", ctypes.c_int64), ("in_dtype", ctypes.c_int),
                ("fp8_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


def _code(dtype, name: str, kinds: str) -> int:
    """The C dtype code; kinds: "w" bf16 and fp32, "8" the 8-bit floats, or both."""
    torch = _torch()
    codes = {}
    if "w" in kinds:
        codes.update({torch.bfloat16: 0, torch.float32: 1})
    if "8" in kinds:
        codes.update({torch.float8_e4m3fn: DORA_E4M3, torch.float8_e5m2: DORA_E5M2})
    if dtype not in codes:
        raise TypeError(f"{name} is {dtype}, expected one of {', '.join(str(d) for d in codes)}")
    return codes[dtype]


def _tensor(t, shape, dtype, device, name: str) -> None:
    """Shape, dtype and device of one tensor (None is skipped): the C ABI cannot see them."""
    if t is None:
        return
    _shape(t, shape, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _current(device) -> None:
    torch = _torch()
    if device.type == "cuda" and device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, but the current device is cuda:{torch.cuda.current_device()}; "
                         f"call under torch.cuda.device({device.index})")


def _on(stream):
    """What is allocated for a call belongs to the stream that uses it."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def dora_fp8_quantize(x, *, block: str = "row", dtype=None, q=None, scale=None, stream=None):
    """(q, scale) of a bf16 or float32 matrix x in blocks of 1 x 128 ("row") or 128 x 128 ("tile").

    Scales are powers of two, [ceil(cols / 128), rows] by row and
    [ceil(rows / 128), ceil(cols / 128)] by tile; dtype is float8_e4m3fn
    (default) or float8_e5m2; cols is a multiple of 16.
    """
    torch = _torch()
    lib = load_library()
    if block not in _BLOCKS:
        raise ValueError(f"block is {block!r}, expected 'row' or 'tile'")
    if x.dim() != 2:
        raise ValueError(f"x has {x.dim()} dimensions, expected 2")
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    code, out = _code(x.dtype, "x", "w"), _code(dtype, "dtype", "8")
    rows, cols = x.shape
    up = lambda n: -(-n // 128)
    shape = (up(cols), rows) if block == "row" else (up(rows), up(cols))
    _current(x.device)
    _tensor(q, (rows, cols), dtype, x.device, "q")
    _tensor(scale, shape, torch.float32, x.device, "scale")
    with _on(stream):
        q = torch.empty(rows, cols, dtype=dtype, device=x.device) if q is None else q
        scale = torch.empty(shape, dtype=torch.float32, device=x.device) if scale is None else scale
    _check(lib.dora_fp8_quantize(rows, cols, code, out, _BLOCKS[block], _ptr(x), _ptr(q), _ptr(scale),
                                 _stream_ptr(stream)))
    return q, scale


def _product(op: int, x, wq, w_scale, x_scale, out, out_dtype, fp8_dtype, ws, stream):
    torch = _torch()
    lib = load_library()
    xn, on = ("x", "y") if op == DORA_FP8_OP_FORWARD else ("dy", "dx")
    if x.dim() != 2 or wq.dim() != 2:
        raise ValueError(f"{xn} and wq are matrices")
    d_out, d_in = wq.shape
    K, N = (d_in, d_out) if op == DORA_FP8_OP_FORWARD else (d_out, d_in)
    T, dev = x.shape[0], x.device
    code = _code(x.dtype, xn, "w8")
    up = lambda n: -(-n // 128)
    _current(dev)
    _tensor(x, (T, K), x.dtype, dev, xn)
    _tensor(wq, (d_out, d_in), torch.float8_e4m3fn, dev, "wq")
    _tensor(w_scale, (up(d_out), up(d_in)), torch.float32, dev, "w_scale")
    if code in (DORA_E4M3, DORA_E5M2):
        if x_scale is None:
            raise ValueError(f"an 8-bit {xn} needs {xn}_scale")
        if out_dtype is None and out is None:
            out_dtype = torch.bfloat16
    elif x_scale is not None:
        raise ValueError(f"{xn}_scale is for an 8-bit {xn}; a {x.dtype} one is quantised in the call")
    _tensor(x_scale, (up(K), T), torch.float32, dev, f"{xn}_scale")
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    ocode = _code(out_dtype, "out_dtype", "w")
    _tensor(out, (T, N), out_dtype, dev, on)
    fcode = _code(torch.float8_e4m3fn if fp8_dtype is None else fp8_dtype, "fp8_dtype", "8")
    desc = Fp8Desc(d_out, d_in, code, fcode, ocode)
    need = int(lib.dora_fp8_workspace_size(ctypes.byref(desc), T, op))
    with _on(stream):
        out = torch.empty(T, N, dtype=out_dtype, device=dev) if out is None else out
        if ws is None and need:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    fn = lib.dora_fp8_forward if op == DORA_FP8_OP_FORWARD else lib.dora_fp8_backward
    _check(fn(ctypes.byref(desc), T, _ptr(x), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(out), _ptr(ws), nbytes,
              _stream_ptr(stream)))
    return out


def dora_fp8_workspace_size(d_out: int, d_in: int, in_dtype, T: int, op: int, *, fp8_dtype=None,
                            out_dtype=None) -> int:
    """Bytes of workspace a product needs (op: DORA_FP8_OP_FORWARD or DORA_FP8_OP_BACKWARD)."""
    torch = _torch()
    code = _code(in_dtype, "in_dtype", "w8")
    out = torch.bfloat16 if out_dtype is None and code > 1 else (in_dtype if out_dtype is None else out_dtype)
    desc = Fp8Desc(int(d_out), int(d_in), code, _code(fp8_dtype or torch.float8_e4m3fn, "fp8_dtype", "8"),
                   _code(out, "out_dtype", "w"))
    return int(load_library().dora_fp8_workspace_size(ctypes.byref(desc), int(T), int(op)))


def dora_fp8_forward(x, wq, w_scale, *, x_scale=None, out_dtype=None, fp8_dtype=None, y=None, ws=None, stream=None):
    """y = x W^T [T, d_out] for a weight held as e4m3 in 128 x 128 blocks.

    x [T, d_in]: bf16 or float32 (quantised in the call to fp8_dtype, e4m3 by
    default), or already 8-bit with x_scale from dora_fp8_quantize(block="row").
    y has out_dtype: x's own, or bf16 for an 8-bit x.
    """
    return _product(DORA_FP8_OP_FORWARD, x, wq, w_scale, x_scale, y, out_dtype, fp8_dtype, ws, stream)


def dora_fp8_backward(dy, wq, w_scale, *, dy_scale=None, out_dtype=None, fp8_dtype=None, dx=None, ws=None,
                      stream=None):
    """dx = dy W [T, d_in], the input gradient of dora_fp8_forward (arguments as there)."""
    return _product(DORA_FP8_OP_BACKWARD, dy, wq, w_scale, dy_scale, dx, out_dtype, fp8_dtype, ws, stream)
