"""The AdamW step and the global gradient norm on the GPU against the float64 oracle.

Bounds, with h = 2^-24 (half a step of fp32): a moment is a sum of two products,
off by at most 4 h of the sum of its terms' magnitudes (three roundings, one of
the gradient's scale). The parameter's update lr1 m / (r rbc2 + eps) adds the
roundings of lr1 and rbc2 (each a few h: expm1f is within one step, its
argument within two half steps, and x e^x / (e^x - 1) <= 1 there), of the root,
of the denominator and of an approximate quotient (two steps): at most 32 h
of its magnitude in all; p - lr wd p and the sum add 4 h of |p|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from oracle import adamw as oa

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
H = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: H}
LR, BETAS, EPS = 3e-3, (0.9, 0.999), 1e-8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64).reshape(-1)


def draw(sizes, dtypes, seed=0, offset=0, std=1.0):
    """Tensors of these sizes; offset > 0 puts each that many elements into a buffer of its own."""
    rng = np.random.default_rng(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.zeros(n + offset + 8, dtype=dtypes[i % len(dtypes)], device="cuda")
        t[offset:offset + n] = torch.from_numpy(rng.standard_normal(n) * std * 10.0 ** rng.uniform(-3, 0)).to(t)
        out.append(t[offset:offset + n])
    return out


class Held:
    """What a handle holds for each tensor, read back in float64."""

    def __init__(self, opt, params, master):
        self.opt, self.params, self.master = opt, params, master
        self.sizes = [-(-p.numel() // 128) * 128 for p in params]

    def read(self):
        s = {k: v for k, v in self.opt.state_dict().items()}
        at = am = 0
        out = []
        for p, size in zip(self.params, self.sizes):
            n = p.numel()
            cut = lambda k: host(s[k][at:at + n])
            e = {"m": cut("avg"), "v": cut("sq"), "at": at}
            if self.opt.state_bits == 8:
                e["cm"], e["cr"] = e["m"], e["v"]
                e["sm"], e["sr"] = (host(s[k][at // 128:(at + size) // 128]) for k in ("avg_scale", "sq_scale"))
                wide = lambda sc: np.repeat(sc, 128)[:n]
                e["m"], e["v"] = e["cm"] * wide(e["sm"]), (e["cr"] * wide(e["sr"])) ** 2
            e["half"] = 0.0 if self.master and p.dtype == BF else HALF[p.dtype]  # the held copy's own rounding
            if self.master and p.dtype == BF:
                e["p"] = host(s["master"][am:am + n])
                am += size
            else:
                e["p"] = host(p)
            out.append(e)
            at += size
        return out


def check_step(before, after, params, grads, t, bits, decay, seed, scale=1.0, lr=LR, betas=BETAS, eps=EPS):
    for i, (b, a, p, g) in enumerate(zip(before, after, params, grads)):
        if p.numel() == 0:
            continue
        gh = host(g)
        rp, rm, rv = oa.step(b["p"], gh, b["m"], b["v"], t, lr=lr, betas=betas, eps=eps, weight_decay=decay[i],
                             scale=scale)
        em = 4 * H * (betas[0] * np.abs(b["m"]) + (1 - betas[0]) * np.abs(scale * gh))
        denom = np.sqrt(rv / (1 - betas[1] ** t)) + eps
        upd = lr / (1 - betas[0] ** t) / denom
        tol = 4 * H * np.abs(b["p"]) + upd * em + 32 * H * np.abs(upd * rm) + 1e-44
        assert np.all(np.abs(a["p"] - rp) <= tol + a["half"] * (np.abs(rp) + tol)), (i, "p")
        assert np.all(np.abs(host(p) - rp) <= tol + HALF[p.dtype] * (np.abs(rp) + tol)), (i, "param")
        if bits == 32:
            assert np.all(np.abs(a["m"] - rm) <= em + 1e-44), (i, "m")
            assert np.all(np.abs(a["v"] - rv) <= 6 * H * rv + 1e-44), (i, "v")
            continue
        r = np.sqrt(rv)
        u = oa.random16(p.numel(), seed, t, b["at"])
        for code, sc, x, zero_up in ((a["cm"], a["sm"], rm, False), (a["cr"], a["sr"], r, True)):
            ex = em if not zero_up else 6 * H * r
            big = oa.blocks(ex).max(axis=1) / 448.0
            assert np.all(np.abs(sc - oa.moment_scale(x)) <= 4 * H * oa.moment_scale(x) + big), (i, "scale")
            want, s = oa.code_steps(x, sc, u)
            got = np.abs(code) / s
            # |y| / s is at most 16 and off by 8 h of itself (and the moment's own error): another code only there
            near = 16 * 8 * H + ex / (np.repeat(sc, 128)[:x.size] * s)
            low, high = np.floor(want - near), np.floor(want + near)
            if zero_up:
                low, high = np.where(x > 0, np.maximum(low, 1), low), np.where(x > 0, np.maximum(high, 1), high)
            assert np.all((got >= low) & (got <= high)), (i, "code", zero_up)
            assert np.all((code == 0) | (np.sign(code) == np.sign(x))), (i, "sign")


SIZES = [1, 7, 8, 16, 127, 128, 129, 2040, 2048, 2049, 5000, 0, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd,gd", [((BF,), (BF,)), ((F32,), (F32,)), ((BF, F32), (F32, BF))])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_steps(bits, pd, gd, master, offset):
    """Three steps over odd sizes, mixed types and odd alignments, each checked from the state before it."""
    params = draw(SIZES, pd, seed=1, offset=offset)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    grads = draw(SIZES, gd, seed=2, offset=offset)
    opt = dw.DoraAdamW(params, grads, lr=LR, betas=BETAS, eps=EPS, weight_decay=decay, state_bits=bits, master=master,
                       seed=77)
    held = Held(opt, params, master)
    for t in (1, 2, 3):
        for g, new in zip(grads, draw(SIZES, gd, seed=2 + t)):
            g.copy_(new)
        before = held.read()
        assert opt.step() is None
        check_step(before, held.read(), params, grads, t, bits, decay, 77)
        assert int(opt.state_dict()["step"]) == t


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_stay(bits):
    """What lies before and behind each parameter is left as it was."""
    bufs = [torch.full((n + 16,), 7.0, dtype=BF, device="cuda") for n in (1, 100, 2047)]
    params = [b[8:8 + n] for b, n in zip(bufs, (1, 100, 2047))]
    opt = dw.DoraAdamW(params, [torch.ones_like(p) for p in params], lr=0.1, state_bits=bits)
    opt.step()
    for b, p in zip(bufs, params):
        assert (b[:8] == 7).all() and (b[8 + p.numel():] == 7).all() and (p != 7).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step(bits):
    sizes = [3000, 129, 17]
    params, grads = draw(sizes, (BF, F32), seed=5), draw(sizes, (BF, F32), seed=6, std=30.0)
    opt = dw.DoraAdamW(params, grads, lr=LR, betas=BETAS, eps=EPS, state_bits=bits, seed=3)
    held = Held(opt, params, False)
    before = held.read()
    norm = opt.step(max_norm=0.5)
    rn, scale = oa.grad_norm([host(g) for g in grads], 0.5)
    assert abs(float(norm) - rn) <= 8 * H * rn
    check_step(before, held.read(), params, grads, 1, bits, [0.0] * 3, 3, scale=float(np.float32(scale)))
    # no clipping below max_norm, and a device scale of the caller's
    before = held.read()
    opt.step(max_norm=1e9)
    check_step(before, held.read(), params, grads, 2, bits, [0.0] * 3, 3)
    before = held.read()
    opt.step(grad_scale=torch.tensor(0.25, device="cuda"))
    check_step(before, held.read(), params, grads, 3, bits, [0.0] * 3, 3, scale=0.25)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bad_gradient_skips_the_step(bits, bad):
    params, grads = draw([500, 3000], (BF,), seed=7), draw([500, 3000], (BF,), seed=8)
    opt = dw.DoraAdamW(params, grads, lr=LR, state_bits=bits, master=True)
    opt.step(max_norm=1.0)
    keep = grads[1][100].clone()
    grads[1][100] = bad
    snap = {k: v.clone() for k, v in opt.state_dict().items()}
    psnap = [p.clone() for p in params]
    norm = opt.step(max_norm=1.0)
    assert not torch.isfinite(norm)
    assert all(torch.equal(v.view(torch.uint8) if v.element_size() == 1 else v, snap[k].view(torch.uint8) if v.element_size() == 1 else snap[k])
               for k, v in opt.state_dict().items())
    assert all(torch.equal(a, b) for a, b in zip(params, psnap))
    grads[1][100] = keep
    opt.step(max_norm=1.0)
    assert int(opt.state_dict()["step"]) == 2


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    sizes = [(i * 37) % 400 + 1 for i in range(1500)]
    params, grads = draw(sizes, (BF,), seed=9), draw(sizes, (BF,), seed=10)
    opt = dw.DoraAdamW(params, grads, lr=LR, betas=BETAS, eps=EPS, state_bits=bits)
    held = Held(opt, params, False)
    before = held.read()
    norm = opt.step(max_norm=1e9)
    rn, _ = oa.grad_norm([host(g) for g in grads])
    assert abs(float(norm) - rn) <= 8 * H * rn
    check_step(before, held.read(), params, grads, 1, bits, [0.0] * len(sizes), 0)
    assert int(opt.state_dict()["step"]) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_replays_further_steps(bits):
    """A captured clipped step, replayed with new gradients and learning rates, gives the eager steps' bits."""
    sizes = [5000, 300, 64]
    res = []
    for captured in (False, True):
        params, grads = draw(sizes, (BF, F32), seed=11), draw(sizes, (BF,), seed=12)
        opt = dw.DoraAdamW(params, grads, lr=LR, state_bits=bits, master=True, seed=5)
        opt.step(max_norm=1.0)
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                opt.step(max_norm=1.0)
        for t in range(4):
            for g, new in zip(grads, draw(sizes, (BF,), seed=20 + t)):
                g.copy_(new)
            opt.set_lr(LR / (t + 1))
            graph.replay() if captured else opt.step(max_norm=1.0)
        torch.cuda.synchronize()
        assert int(opt.state_dict()["step"]) == 5
        res.append([p.clone() for p in params] + [v.clone().view(torch.uint8) for k, v in opt.state_dict().items() if k != "step"])
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("sizes", [[3000, 50], [(i * 53) % 900 + 1 for i in range(800)]])
@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_in_the_step_and_before_it_agree(sizes, bits):
    """step(max_norm=) gives the bits of grad_norm(max_norm) followed by step(grad_scale=)."""
    res = []
    for fused in (True, False):
        params, grads = draw(sizes, (BF, F32), seed=30), draw(sizes, (BF,), seed=31, std=3.0)
        opt = dw.DoraAdamW(params, grads, lr=LR, state_bits=bits, seed=2)
        for _ in range(2):
            if fused:
                norm = opt.step(max_norm=0.7)
            else:
                norm, scale = opt.grad_norm(0.7)
                opt.step(grad_scale=scale)
        res.append([norm] + params + [v.clone().view(torch.uint8) for k, v in opt.state_dict().items() if k != "step"])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_saved_state_continues():
    params, grads = draw([3000, 50], (BF,), seed=13), draw([3000, 50], (BF,), seed=14)
    a = dw.DoraAdamW(params, grads, lr=LR, state_bits=8, master=True, seed=9)
    for _ in range(3):
        a.step()
    copies = [p.clone() for p in params]
    b = dw.DoraAdamW(copies, grads, lr=LR, state_bits=8, master=True, seed=9)
    b.load_state_dict({k: v.clone() for k, v in a.state_dict().items()})
    a.step()
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(params, copies))
    assert torch.equal(a.state_dict()["avg"].view(torch.uint8), b.state_dict()["avg"].view(torch.uint8))
    with pytest.raises(KeyError):
        a.load_state_dict({"nothing": copies[0]})
    with pytest.raises(ValueError, match="avg"):
        a.load_state_dict({"avg": torch.zeros(3, device="cuda")})


def test_eight_bit_moments_follow_the_mean():
    """Beside a neighbour 40 times larger, a gradient of 1 from a zero state: sqrt(v) has to climb by fractions of a code
    per step. After 600 steps v = 1 - 0.999^600 = 0.451. A code's spacing is at most 1/8 of its value, so the
    rounding of one step moves sqrt(v) by a variance of at most (1/8)^2 / 4 of its square; the noise decays
    with the moment (by 0.9995 a step), so its standard deviation is at most sqrt(1 / 256 / 0.001) = 2 of one
    value in the worst case, 0.05 of the mean over 1600; its square biases v upward. Nearest rounding would leave
    v near 0.02. The bounds are a quarter and four times."""
    n = 128 * 16
    p = torch.zeros(n, device="cuda")
    g = torch.ones(n, device="cuda")
    g[::128] = 40.0
    opt = dw.DoraAdamW([p], [g], lr=0.0, state_bits=8, seed=1)
    for _ in range(600):
        opt.step()
    s = opt.state_dict()
    v = (host(s["sq"]).reshape(-1, 128) * host(s["sq_scale"])[:, None]) ** 2
    m = host(s["avg"]).reshape(-1, 128) * host(s["avg_scale"])[:, None]
    assert 0.451 / 4 <= v[:, 1:].mean() <= 4 * 0.451
    assert abs(v[:, 0].mean() / 1600 - 0.451) <= 0.451 * 0.01  # the largest of a block has the scale to itself
    assert abs(m[:, 1:].mean() - 1.0) <= 0.05
    assert (p == 0).all()


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("sizes", [[1], [8], [5, 2049, 128], [300000], [(i * 91) % 3000 for i in range(2300)]])
@pytest.mark.parametrize("dt", [(BF,), (F32,), (F32, BF)])
def test_grad_norm(sizes, dt):
    grads = draw(sizes, dt, seed=15, offset=1)
    norm, scale = dw.dora_grad_norm(grads, 2.0)
    rn, rs = oa.grad_norm([host(g) for g in grads], 2.0)
    # eight squares and their sums in fp32 (8 h of a sum of positives, halved by the root), one rounding
    assert abs(float(norm) - rn) <= 6 * H * rn
    assert abs(float(scale) - rs) <= 8 * H * rs
    again, _ = dw.dora_grad_norm(grads, 2.0)
    assert torch.equal(norm, again)


def test_grad_norm_range():
    """Squares that overflow or vanish in fp32 do not: the norm is right over the range of the type."""
    for v in (1e30, 1e-30, 3e38):
        g = torch.full((1000,), v, device="cuda")
        norm, scale = dw.dora_grad_norm([g], 1.0)
        want = v * np.sqrt(1000.0)
        if want > 3.4e38:
            assert torch.isinf(norm)
        else:
            assert abs(float(norm) / (float(np.float32(v)) * np.sqrt(1000.0)) - 1) <= 6 * H
    norm, scale = dw.dora_grad_norm([torch.zeros(50, device="cuda")], 1.0)
    assert float(norm) == 0 and float(scale) == 1
    norm, scale = dw.dora_grad_norm([torch.empty(0, device="cuda")])
    assert float(norm) == 0 and float(scale) == 1
