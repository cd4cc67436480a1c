"""Shared by the GPU tests of the 8-bit products: operands, the calls, and the bounds against float64.

Bounds: the tensor cores' accumulator adds 128 exact products of a block (scales that are no powers of two, or an fp32
result of more than 32 blocks), or all K of them (powers of two), each addition off by at most 2^-23 of the sum of
|products|; folding nkb blocks adds (nkb + 3) * 2^-24 of it; the result is rounded once. As independent roundings the
sums are off by about sqrt(sums) * 2^-24 and the folds by sqrt(nkb) * 2^-24 of the partial sums, so the whole matrix is
held to (sqrt(sums) + sqrt(nkb)) * 2^-22 of its norm.
"""
import numpy as np
import torch

import dora_weight_decomposed_b200 as dw
from oracle import fp8 as of

BF, F32, E4, E5 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
NAME = {E4: "e4m3", E5: "e5m2"}


def launches(call):
    """The kernels that a call launches, by their names."""
    dw.dora_profile_start(16)
    try:
        call()
        return [n for n, _ in dw.dora_profile_read()]
    finally:
        dw.dora_profile_stop()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(rows, cols, fp8, seed):
    """Codes of normal values, clamped into the type's range: no NaN among them."""
    top = of.TOP[NAME[fp8]]
    return (torch.randn(rows, cols, generator=gen(seed), device="cuda") * top / 4).clamp(-top, top).to(fp8)


def scales(rows, cols, seed, powers, lo=-10, hi=10):
    if powers:
        return torch.exp2(torch.randint(lo, hi, (rows, cols), generator=gen(seed), device="cuda").float())
    return torch.rand(rows, cols, generator=gen(seed), device="cuda") * 3 + 0.01


def wide_rows(q, s):
    return q.double() * s.double().T.repeat_interleave(128, 1)[:, :q.shape[1]]


def wide_tiles(q, s):
    return q.double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def blocks(n):
    return -(-n // 128)


def call(backward, x, wq, ws, xs=None, out=None, **kw):
    if xs is not None:
        kw["dy_scale" if backward else "x_scale"] = xs
    if out is not None:
        kw["dx" if backward else "y"] = out
    return (dw.dora_fp8_backward if backward else dw.dora_fp8_forward)(x, wq, ws, **kw)


def check(out, x, w, K, whole):
    """out against x @ w in float64; whole: all K products of a result may have been added in one accumulator."""
    ref, mag = x @ w, x.abs() @ w.abs()
    sums, nkb = (K if whole else 128), blocks(K)
    tol = (sums * 2.0 ** -23 + (nkb + 3) * 2.0 ** -24) * mag
    tol = tol + HALF[out.dtype] * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp_min(1e-300)).max())
    far = float(torch.linalg.norm(out.double() - ref) / torch.linalg.norm(ref))
    assert far <= (np.sqrt(sums) + np.sqrt(nkb)) * 2.0 ** -22 + HALF[out.dtype], far
