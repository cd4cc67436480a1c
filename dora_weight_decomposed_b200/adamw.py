"""The update of the trained tensors: global gradient norm and AdamW over many tensors.

    opt = DoraAdamW([A0, B0, m0, A1, ...], [dA0, dB0, dm0, dA1, ...], lr=1e-4, state_bits=8, master=True)
    ...                                    # dora_backward(..., dm=dm0, dA=dA0, dB=dB0), dp.allreduce_gradients
    norm = opt.step(max_norm=1.0)

The handle binds the parameters and the gradient buffers once: gradients are
written into the same buffers every step (dora_backward's dm=, dA=, dB=), and a
step is a single call into the library that reads them where they lie. The step
count and the learning rate live in device memory, so a step captured in a CUDA
graph replays as further steps. See include/dora.h for the formulas.
"""
from __future__ import annotations

import ctypes
import math

from . import _check, _ptr, _torch, load_library
from .fp8 import _WIDE, _code, _current, _empty, _stream


class GradEntry(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("scale_avg", ctypes.c_void_p), ("scale_sq", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("numel", ctypes.c_int64), ("index0", ctypes.c_int64),
                ("weight_decay", ctypes.c_float), ("param_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int)]


class AdamwDesc(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_float),
                ("state_bits", ctypes.c_int), ("seed", ctypes.c_uint32)]


def _grad_table(grads, device):
    for i, g in enumerate(grads):
        if g.device != device:
            raise ValueError(f"gradient {i} is on {g.device}, expected {device}")
    return (GradEntry * max(len(grads), 1))(*[GradEntry(_ptr(g), g.numel(), _code(g.dtype, f"gradient {i}", _WIDE))
                                              for i, g in enumerate(grads)])


def _grad_norm(table, n: int, max_norm: float, ws, device, stream):
    torch, lib = _torch(), load_library()
    norm, scale = (_empty((), torch.float32, device, stream) for _ in range(2))
    if ws is None:
        ws = _empty(int(lib.dora_grad_norm_workspace_size(n)), torch.uint8, device, stream)
    _check(lib.dora_grad_norm(table, n, max_norm, norm.data_ptr(), scale.data_ptr(), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream, device)))
    return norm, scale


def dora_grad_norm(grads, max_norm: float = math.inf, *, ws=None, stream=None):
    """(norm, scale) of the gradients taken together, two float32 scalars on the device.

    norm = sqrt(sum of squares over all tensors); scale = min(1, max_norm /
    (norm + 1e-6)), NaN when the norm is not finite (DoraAdamW.step then skips).
    """
    grads = list(grads)
    if not grads:
        raise ValueError("grads is empty")
    device = grads[0].device
    _current(device)
    if ws is not None and ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    return _grad_norm(_grad_table(grads, device), len(grads), float(max_norm), ws, device, stream)


class DoraAdamW:
    """AdamW over a fixed list of parameters and gradient buffers.

    params, grads: contiguous bf16 or float32 tensors of equal shapes (types may
        differ), all on one device; parameters must not overlap. The handle
        keeps them alive and uses their storage as it is now.
    lr, betas, eps, weight_decay: as usual; weight_decay may be a list.
    state_bits: 32, or 8 (e4m3 codes with one scale per 128 elements, rounded
        stochastically from `seed`).
    master: keep a float32 copy of every bf16 parameter and round the parameter
        from it; without it a bf16 parameter loses updates under half its spacing.

    The state is made on the current stream: a step on another one is ordered
    behind that by the caller, who also keeps the handle until its steps are done.
    """

    def __init__(self, params, grads, *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0,
                 state_bits: int = 32, master: bool = False, seed: int = 0):
        torch = _torch()
        params, grads = [p.detach() for p in params], [g.detach() for g in grads]
        if not params or len(params) != len(grads):
            raise ValueError(f"{len(params)} parameters and {len(grads)} gradients")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits is {state_bits}, expected 8 or 32")
        n = len(params)
        decay = [float(w) for w in weight_decay] if hasattr(weight_decay, "__len__") else [float(weight_decay)] * n
        if len(decay) != n:
            raise ValueError(f"{len(decay)} weight decays for {n} parameters")
        device = params[0].device
        _current(device)
        for i, (p, g) in enumerate(zip(params, grads)):
            if p.shape != g.shape:
                raise ValueError(f"gradient {i} has shape {tuple(g.shape)}, expected {tuple(p.shape)}")
            if p.device != device:
                raise ValueError(f"parameter {i} is on {p.device}, expected {device}")
            _code(p.dtype, f"parameter {i}", _WIDE)
        self._grads = _grad_table(grads, device)
        spans = sorted((_ptr(p), p.numel() * p.element_size(), i) for i, p in enumerate(params) if p.numel())
        for (a, size, i), (b, _, j) in zip(spans, spans[1:]):
            if a + size > b:
                raise ValueError(f"parameters {i} and {j} overlap")

        # State of all tensors in flat buffers, each tensor's part padded to whole blocks of 128.
        sizes = [-(-p.numel() // 128) * 128 for p in params]
        total = sum(sizes)
        self.state_bits = state_bits
        f32 = dict(dtype=torch.float32, device=device)
        moment = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        self._state = {"avg": torch.zeros(total, dtype=torch.float32, device=device).to(moment),
                       "sq": torch.zeros(total, dtype=torch.float32, device=device).to(moment)}
        if state_bits == 8:
            self._state["avg_scale"] = torch.zeros(total // 128, **f32)
            self._state["sq_scale"] = torch.zeros(total // 128, **f32)
        if master:
            self._state["master"] = torch.zeros(
                sum(s for s, p in zip(sizes, params) if p.dtype == torch.bfloat16), **f32)
        self._control = torch.zeros(2, dtype=torch.int64, device=device)  # step, then lr and a counter
        self._lr = self._control.view(torch.float32)[2:3]
        self.set_lr(lr)
        self._desc = AdamwDesc(float(betas[0]), float(betas[1]), float(eps), int(state_bits), int(seed) & 0xFFFFFFFF)
        width = 4 if state_bits == 32 else 1
        base = {k: v.data_ptr() for k, v in self._state.items()}
        rows, at, at_master = [], 0, 0
        for i, (p, g, size) in enumerate(zip(params, grads, sizes)):
            held = master and p.dtype == torch.bfloat16
            if held:
                self._state["master"][at_master:at_master + p.numel()].copy_(p.reshape(-1))
            rows.append(AdamwTensor(
                _ptr(p), _ptr(g), base["avg"] + at * width, base["sq"] + at * width,
                base["avg_scale"] + at // 32 if state_bits == 8 else None,
                base["sq_scale"] + at // 32 if state_bits == 8 else None,
                base["master"] + at_master * 4 if held else None, p.numel(), at, decay[i],
                _code(p.dtype, f"parameter {i}", _WIDE), _code(g.dtype, f"gradient {i}", _WIDE)))
            at += size
            at_master += size if held else 0
        self._tensors = (AdamwTensor * n)(*rows)
        self._n, self._device, self._keep = n, device, (params, grads)
        self._ref, self._control_ptr = ctypes.byref(self._desc), self._control.data_ptr()
        # The partial sums that a clipped step keeps between its kernels.
        self._ws_bytes = int(load_library().dora_grad_norm_workspace_size(n))
        self._ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=device)
        self._ws_ptr = self._ws.data_ptr()

    def set_lr(self, lr: float) -> None:
        """The learning rate of the steps queued from now on (written on the current stream)."""
        if not (math.isfinite(lr) and lr >= 0.0):
            raise ValueError(f"lr is {lr}")
        self._lr.fill_(float(lr))

    def grad_norm(self, max_norm: float = math.inf, *, stream=None):
        """dora_grad_norm of the bound gradients (with a workspace of its own: it may run beside a step)."""
        _current(self._device)
        return _grad_norm(self._grads, self._n, float(max_norm), None, self._device, stream)

    def step(self, *, max_norm: float | None = None, grad_scale=None, stream=None):
        """One step from the bound gradients; returns their norm when max_norm is given.

        max_norm clips by the global norm; grad_scale is instead a float32
        scalar tensor on the device that multiplies the gradients. A scale that
        is not finite (a non-finite norm among them) skips the step.
        """
        torch = _torch()
        device = self._device
        _current(device)
        lib = load_library()
        if max_norm is not None:
            if grad_scale is not None:
                raise ValueError("give max_norm or grad_scale, not both")
            norm = self._lr.new_empty(()) if stream is None else _empty((), torch.float32, device, stream)
            _check(lib.dora_adamw_clipped(self._ref, self._tensors, self._n, self._control_ptr, max_norm, norm.data_ptr(),
                                          self._ws_ptr, self._ws_bytes, _stream(stream, device)))
            return norm
        if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or
                                       grad_scale.device != device):
            raise ValueError(f"grad_scale must be one float32 value on {device}")
        _check(lib.dora_adamw(self._ref, self._tensors, self._n, self._control_ptr, _ptr(grad_scale),
                              _stream(stream, device)))
        return None

    def state_dict(self) -> dict:
        """The live state: flat moments (8 bits: codes and scales), the master copy, the step count (int64 tensor)."""
        return {**self._state, "step": self._control[0]}

    def load_state_dict(self, state: dict) -> None:
        """Copy a state_dict (or part of one) in; "step" may be an int. A master copy does not change the parameters.

        A state that is refused leaves the handle as it was.
        """
        step = None
        for k, v in state.items():
            if k == "step":
                step = int(v)
                if step < 0:
                    raise ValueError(f"step is {step}")
                continue
            if k not in self._state:
                raise KeyError(f"no state {k!r} here (have {sorted(self._state)})")
            mine = self._state[k]
            if v.shape != mine.shape or v.dtype != mine.dtype:
                raise ValueError(f"{k} is {v.dtype} {tuple(v.shape)}, expected {mine.dtype} {tuple(mine.shape)}")
        for k, v in state.items():
            if k != "step":
                self._state[k].copy_(v)
        if step is not None:
            self._control[0].fill_(step)
