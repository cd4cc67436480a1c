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

import ctypes
import functools

from . import _check, _ptr, _shape, _stream_ptr, _torch, load_library

DORA_E4M3, DORA_E5M2 = 2, 3
DORA_FP8_OP_FORWARD, DORA_FP8_OP_BACKWARD = 0, 1
_BLOCKS = {"row": 0, "tile": 1}


class Fp8Desc(ctypes.Structure):
    _fields_ = [("d_out", ctypes.c_int64), ("d_in", ctypes.c_int64), ("in_dtype", ctypes.c_int),
                ("fp8_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


_WIDE: dict = {}   # dtype -> C code, filled on first use (torch is imported late)
_EIGHT: dict = {}
_BOTH: dict = {}


def _codes() -> None:
    torch = _torch()
    _WIDE.update({torch.bfloat16: 0, torch.float32: 1})
    _EIGHT.update({torch.float8_e4m3fn: DORA_E4M3, torch.float8_e5m2: DORA_E5M2})
    _BOTH.update({**_WIDE, **_EIGHT})


def _code(dtype, name: str, among: dict) -> int:
    """The C dtype code, of the types in `among`."""
    if not _BOTH:
        _codes()
    code = among.get(dtype)
    if code is None:
        raise TypeError(f"{name} is {dtype}, expected one of {', '.join(str(d) for d in among)}")
    return code


def _tensor(t, shape, dtype, device, name: str) -> None:
    """Shape, dtype and device of one tensor: the C ABI cannot see them."""
    if t.shape != shape:
        _shape(t, shape, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


_current_device = None  # index of the current device: torch.cuda.current_device, or what it calls, set on first use


def _current(device) -> None:
    global _current_device
    if device.type == "cuda":
        if _current_device is None:
            torch = _torch()
            torch.cuda.current_device()  # CUDA is initialised from here on
            _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        if device.index != _current_device():
            raise ValueError(f"tensors are on {device}, but the current device is cuda:{_current_device()}; "
                             f"call under torch.cuda.device({device.index})")


_raw_stream = None  # device index -> handle of its current stream, set on first use


def _stream(stream, device):
    """_stream_ptr, without building a stream object for the current stream (a third of a small call's host time)."""
    global _raw_stream
    if stream is None and device.type == "cuda":
        if _raw_stream is None:
            torch = _torch()
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda index: torch.cuda.current_stream(index).cuda_stream)
        return _raw_stream(device.index) or None
    return _stream_ptr(stream)


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream that uses it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def dora_fp8_quantize(x, *, block: str = "row", dtype=None, q=None, scale=None, stream=None):
    """(q, scale) of a bf16 or float32 matrix x in blocks of 1 x 128 ("row") or 128 x 128 ("tile").

    Scales are powers of two, [ceil(cols / 128), rows] by row and
    [ceil(rows / 128), ceil(cols / 128)] by tile; dtype is float8_e4m3fn
    (default) or float8_e5m2; cols is a multiple of 16.
    """
    sig = (block, x.shape, x.dtype, dtype)
    plan = _QUANTIZE_PLANS.get(sig) or _quantize_plan(sig, x)
    code, out, how, shape, qtype, call = plan
    dev = x.device
    _current(dev)
    f32 = _torch().float32
    if q is None:
        q = x.new_empty(x.shape, dtype=qtype) if stream is None else _empty(x.shape, qtype, dev, stream)
    else:
        _tensor(q, x.shape, qtype, dev, "q")
    if scale is None:
        scale = x.new_empty(shape, dtype=f32) if stream is None else _empty(shape, f32, dev, stream)
    else:
        _tensor(scale, shape, f32, dev, "scale")
    _check(call(x.shape[0], x.shape[1], code, out, how, _ptr(x), _ptr(q), _ptr(scale), _stream(stream, dev)))
    return q, scale


_QUANTIZE_PLANS: dict = {}


def _quantize_plan(sig, x):
    """Check one signature; (code of x, code of q, block, shape of the scales, type of q, library call)."""
    torch = _torch()
    block, _, xtype, dtype = sig
    if block not in _BLOCKS:
        raise ValueError(f"block is {block!r}, expected 'row' or 'tile'")
    if x.dim() != 2:
        raise ValueError(f"x has {x.dim()} dimensions, expected 2")
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    code, out = _code(xtype, "x", _WIDE), _code(dtype, "dtype", _EIGHT)
    rows, cols = x.shape
    shape = (-(-cols // 128), rows) if block == "row" else (-(-rows // 128), -(-cols // 128))
    if len(_QUANTIZE_PLANS) > 4096:
        _QUANTIZE_PLANS.clear()
    plan = _QUANTIZE_PLANS[sig] = (code, out, _BLOCKS[block], shape, dtype, load_library().dora_fp8_quantize)
    return plan


@functools.lru_cache(maxsize=4096)
def _desc_and_workspace(d_out: int, d_in: int, in_code: int, fp8_code: int, out_code: int, T: int, op: int, device):
    """The C descriptor of these sizes and types (a byref of it) and the workspace they need on the current device
    (`device` is its index)."""
    desc = Fp8Desc(d_out, d_in, in_code, fp8_code, out_code)
    ref = ctypes.byref(desc)
    return ref, int(load_library().dora_fp8_workspace_size(ref, T, op))


_PLANS: dict = {}  # what a product of these shapes, types and devices needs: checked once, by signature


def _plan(sig, op: int, x, wq, w_scale, x_scale, out, out_dtype, fp8_dtype):
    """Check one signature; (descriptor, workspace bytes, 8-bit operand?, shape of the result, its type, library call)."""
    torch = _torch()
    lib = load_library()
    xn = "x" if op == DORA_FP8_OP_FORWARD else "dy"
    if x.dim() != 2 or wq.dim() != 2:
        raise ValueError(f"{xn} and wq are matrices")
    d_out, d_in = wq.shape
    K, N = (d_in, d_out) if op == DORA_FP8_OP_FORWARD else (d_out, d_in)
    T, dev, dtype = x.shape[0], x.device, x.dtype
    code = _code(dtype, xn, _BOTH)
    _tensor(x, (T, K), dtype, dev, xn)
    _tensor(wq, (d_out, d_in), torch.float8_e4m3fn, dev, "wq")
    _tensor(w_scale, (-(-d_out // 128), -(-d_in // 128)), torch.float32, dev, "w_scale")
    given = code in (DORA_E4M3, DORA_E5M2)
    if given and x_scale is None:
        raise ValueError(f"an 8-bit {xn} needs {xn}_scale")
    if not given and x_scale is not None:
        raise ValueError(f"{xn}_scale is for an 8-bit {xn}; a {dtype} one is quantised in the call")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16 if given else dtype
    fcode = DORA_E4M3 if fp8_dtype is None else _code(fp8_dtype, "fp8_dtype", _EIGHT)
    _current(dev)
    ref, need = _desc_and_workspace(d_out, d_in, code, fcode, _code(out_dtype, "out_dtype", _WIDE), T, op, dev.index)
    plan = (ref, need, given, (T, N), out_dtype, lib.dora_fp8_forward if op == DORA_FP8_OP_FORWARD else lib.dora_fp8_backward)
    if len(_PLANS) > 4096:
        _PLANS.clear()
    _PLANS[sig] = plan
    return plan


def _product(op: int, x, wq, w_scale, x_scale, out, out_dtype, fp8_dtype, ws, stream):
    sig = (op, x.shape, x.dtype, x.device, wq.shape, wq.dtype, wq.device, w_scale.shape, w_scale.dtype, w_scale.device,
           x_scale is None, out_dtype, fp8_dtype, None if out is None else out.dtype)
    plan = _PLANS.get(sig) or _plan(sig, op, x, wq, w_scale, x_scale, out, out_dtype, fp8_dtype)
    ref, need, given, shape, out_dtype, call = plan
    dev = sig[3]
    _current(dev)
    if given:
        _tensor(x_scale, (-(-x.shape[1] // 128), shape[0]), _torch().float32, dev, "x_scale" if op == DORA_FP8_OP_FORWARD else "dy_scale")
    if out is None:
        out = x.new_empty(shape, dtype=out_dtype) if stream is None else _empty(shape, out_dtype, dev, stream)
    else:
        _tensor(out, shape, out_dtype, dev, "y" if op == DORA_FP8_OP_FORWARD else "dx")
    nbytes = need
    if ws is not None:
        if ws.device != dev:
            raise ValueError(f"ws is on {ws.device}, expected {dev}")
        nbytes = ws.numel() * ws.element_size()
    elif need:
        ws = w_scale.new_empty(-(-need // 4)) if stream is None else _empty(need, _torch().uint8, dev, stream)
    if x.is_cuda and x.is_contiguous() and wq.is_contiguous() and w_scale.is_contiguous():  # all on one device, by the plan
        status = call(ref, shape[0], x.data_ptr(), _ptr(x_scale), wq.data_ptr(), w_scale.data_ptr(), _ptr(out), _ptr(ws),
                      nbytes, _stream(stream, dev))
    else:  # the message of the one that is refused
        status = call(ref, shape[0], _ptr(x), _ptr(x_scale), _ptr(wq), _ptr(w_scale), _ptr(out), _ptr(ws), nbytes,
                      _stream(stream, dev))
    if status:
        _check(status)
    return out


def dora_fp8_workspace_size(d_out: int, d_in: int, in_dtype, T: int, op: int, *, fp8_dtype=None,
                            out_dtype=None) -> int:
    """Bytes of workspace a product needs (op: DORA_FP8_OP_FORWARD or DORA_FP8_OP_BACKWARD)."""
    torch = _torch()
    code = _code(in_dtype, "in_dtype", _BOTH)
    out = torch.bfloat16 if out_dtype is None and code > 1 else (in_dtype if out_dtype is None else out_dtype)
    return _desc_and_workspace(int(d_out), int(d_in), code, _code(fp8_dtype or torch.float8_e4m3fn, "fp8_dtype", _EIGHT),
                               _code(out, "out_dtype", _WIDE), int(T), int(op),
                               torch.cuda.current_device() if torch.cuda.is_available() else None)[1]


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
