"""The AdamW step at the ends of fp32's range: squares of gradients that are subnormal, norms beyond the type.

Bounds, with h = 2^-24: v' = beta2 v + (1 - beta2) g'^2 takes at most eight roundings of h (two of them of a moment
held in 8 bits, which is squared), and each of its terms, squares and sums may be subnormal and is then off by half the
spacing, 2^-150: |v' - v| <= 8 h v + 2^-147. The root and everything behind it are normal numbers here, so the update
adds 40 h of its magnitude to what that leaves of the root.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from oracle import adamw as oa
from oracle import fp8 as of

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
H = 2.0 ** -24
LR, B1, B2 = 3e-3, 0.9, 0.999


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64).reshape(-1)


def gradients(sizes, n, seed):
    """n values of these magnitudes in turn, in blocks of 128 of one magnitude, and in the last blocks mixed."""
    rng = np.random.default_rng(seed)
    mag = np.repeat(np.resize(sizes, -(-n // 128)), 128)[:n]
    mag[-512:] = np.resize(sizes, 512)
    return rng.uniform(0.5, 1.0, n) * rng.choice([-1.0, 1.0], n) * mag


SMALL = [1e-17, 1e-18, 3e-19, 1e-19, 3e-20, 1e-20]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-20])
@pytest.mark.parametrize("gd", [BF, F32])
@pytest.mark.parametrize("sizes", [SMALL, SMALL + [1e-3]])
@pytest.mark.parametrize("offset", [0, 1])
def test_gradients_whose_squares_are_subnormal(bits, eps, gd, sizes, offset):
    n = 2048 + 2048 + 700
    g = torch.zeros(n + offset + 8, dtype=gd, device="cuda")[offset:offset + n]
    g.copy_(torch.from_numpy(gradients(sizes, n, 1)))
    p = torch.zeros(n + offset + 8, device="cuda")[offset:offset + n]
    opt = dw.DoraAdamW([p], [g], lr=LR, betas=(B1, B2), eps=eps, state_bits=bits, seed=3)
    for t in (1, 2):
        s = opt.state_dict()
        m, v, p0, gh = host(s["avg"])[:n], host(s["sq"])[:n], host(p), host(g)
        if bits == 8:
            wide = lambda k: np.repeat(host(s[k]), 128)[:n]
            m, v = m * wide("avg_scale"), (v * wide("sq_scale")) ** 2
        opt.step()
        rp, rm, rv = oa.step(p0, gh, m, v, t, lr=LR, betas=(B1, B2), eps=float(np.float32(eps)), weight_decay=0.0)
        dv = 8 * H * rv + 2.0 ** -147
        low, high = np.sqrt(np.maximum(rv - dv, 0.0)), np.sqrt(rv + dv)
        got_v = host(s["sq"])[:n]
        if bits == 32:
            assert np.all(np.abs(got_v - rv) <= dv)
        else:
            sc = np.repeat(host(s["sq_scale"]), 128)[:n]
            step = of.spacing(got_v, "e4m3") * sc  # a code is the one below or above the root (or the least one)
            assert np.all((got_v > 0) & (np.abs(got_v * sc - np.sqrt(rv)) <= step + (high - low) + 16 * H * high))
            top = oa.blocks(high).max(axis=1) / 448.0
            assert np.all((host(s["sq_scale"]) <= top * (1 + 8 * H)) &
                          (host(s["sq_scale"]) >= oa.blocks(low).max(axis=1) / 448.0 * (1 - 8 * H)))
        if eps == 0.0 and np.any(low == 0.0):
            raise AssertionError("a gradient of this test is too small for a bound")
        u = LR / (1 - B1 ** t) * np.abs(rm)
        den = lambda r: r / np.sqrt(1 - B2 ** t) + float(np.float32(eps))
        em = 4 * H * (B1 * np.abs(m) + (1 - B1) * np.abs(gh))
        tol = 4 * H * np.abs(p0) + LR / (1 - B1 ** t) * em / den(low) + u * (1 / den(low) - 1 / den(high)) + 40 * H * u / den(low)
        assert np.all(np.abs(host(p) - rp) <= tol), np.max(np.abs(host(p) - rp) / tol)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_among_tiny_ones(bits):
    """A zero moment stays zero and its parameter where it is, beside neighbours of any size."""
    n = 4096 + 100
    g = torch.from_numpy(gradients(SMALL + [1e-3], n, 2)).float().cuda()
    g[::3] = 0
    p = torch.ones(n, device="cuda")
    opt = dw.DoraAdamW([p], [g], lr=LR, eps=1e-20, state_bits=bits)
    for _ in range(2):
        opt.step()
    s = opt.state_dict()
    assert (p[::3] == 1).all() and (host(s["sq"])[:n:3] == 0).all() and (host(s["avg"])[:n:3] == 0).all()
    assert (p[1::3] != 1).all() and (host(s["sq"])[1:n:3] > 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_norm_beyond_the_type_skips_the_step(bits):
    """The norm of 1000 gradients of 3e38 is 9.5e39: it is returned as infinite, so it counts as infinite."""
    g = torch.full((1000,), 3e38, device="cuda")
    norm, scale = dw.dora_grad_norm([g], 1.0)
    assert torch.isinf(norm) and torch.isnan(scale)
    p = torch.ones(1000, device="cuda")
    opt = dw.DoraAdamW([p], [g], lr=LR, state_bits=bits)
    assert torch.isinf(opt.step(max_norm=1.0))
    assert (p == 1).all() and int(opt.state_dict()["step"]) == 0
    g.mul_(0.01)  # 9.5e37, inside the type
    norm, scale = dw.dora_grad_norm([g], 1.0)
    assert abs(float(norm) / (float(g[0]) * np.sqrt(1000.0)) - 1) <= 6 * H and float(scale) > 0
    assert torch.isfinite(opt.step(max_norm=1.0)) and (p != 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_moment_that_is_not_finite(bits):
    """A gradient of 3e19 has an infinite square. In 32 bits its element stands still from then on; in 8 bits its block of
    128 shares the scale, and is NaN from the next step on. Every other block goes on as without it."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    g0 = torch.randn(4096, generator=gen, device="cuda")
    res = []
    for bad in (False, True):
        p, g = torch.ones(4096, device="cuda"), g0.clone()
        if bad:
            g[2100] = 3e19
        opt = dw.DoraAdamW([p], [g], lr=LR, state_bits=bits, seed=1)
        opt.step()
        first = p.clone()
        assert bool(torch.isfinite(first).all())
        g.copy_(g0)
        opt.step()
        res.append((first, p))
    (f0, p0), (f1, p1) = res
    keep = torch.ones(4096, dtype=torch.bool, device="cuda")
    keep[2048:2176] = False
    assert torch.equal(p0[keep], p1[keep]) and float(f1[2100]) == 1.0
    if bits == 32:
        assert float(p1[2100]) == 1.0
        keep = torch.ones(4096, dtype=torch.bool, device="cuda")
        keep[2100] = False
        assert torch.equal(p0[keep], p1[keep])
    else:
        assert bool(torch.isnan(p1[2048:2176]).all())
