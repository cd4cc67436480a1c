"""The AdamW step and the gradient norm on a tensor of more than 2^31 elements: its ends against the oracle. The bounds
are those of the short tensors: 4 h (h = 2^-24) of the sum of a moment's terms, 32 h of the update, 4 h of |p|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dora_weight_decomposed_b200 as dw
from oracle import adamw as oa

pytestmark = pytest.mark.gpu
H = 2.0 ** -24
LR, B1, B2, EPS = 3e-3, 0.9, 0.999, 1e-8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dora_weight_decomposed_b200 import build
    build.build()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("clip", [False, True])
def test_offsets_beyond_32_bits(bits, clip):
    if torch.cuda.mem_get_info()[0] < 70e9:
        pytest.skip("needs 70 GB")
    n = 2 ** 31 + 128 * 1001 + 5  # neither a whole chunk nor a whole block at the end
    gen = torch.Generator(device="cuda").manual_seed(4)
    g = torch.randn(n, generator=gen, device="cuda", dtype=torch.bfloat16)
    p = torch.randn(n, generator=gen, device="cuda", dtype=torch.bfloat16)
    opt = dw.DoraAdamW([p], [g], lr=LR, betas=(B1, B2), eps=EPS, state_bits=bits, seed=77)
    s = opt.state_dict()
    norm64 = sum(float((v.float() ** 2).sum(dtype=torch.float64)) for v in g.split(1 << 28)) ** 0.5
    cuts = [slice(0, 4096), slice(2 ** 31 - 2048, 2 ** 31 + 2048), slice(n - 4096 - 5, n)]  # starts are whole blocks
    assert all(c.start % 128 == 0 for c in cuts)
    before = [host(p[c]) for c in cuts]
    norm = opt.step(max_norm=0.5 if clip else None)
    scale = 0.5 / (norm64 + 1e-6) if clip else 1.0
    if clip:
        assert abs(float(norm) - norm64) <= 8 * H * norm64
    for c, p0 in zip(cuts, before):
        gh = host(g[c])
        rp, rm, rv = oa.step(p0, gh, 0.0, 0.0, 1, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.0, scale=scale)
        em = 8 * H * (1 - B1) * np.abs(scale * gh)  # 4 h of the scale itself: it comes from a norm in fp32 squares
        upd = LR / (1 - B1) / (np.sqrt(rv / (1 - B2)) + EPS)
        tol = 4 * H * np.abs(p0) + upd * em + 40 * H * np.abs(upd * rm)
        assert np.all(np.abs(host(p[c]) - rp) <= tol + 2.0 ** -8 * (np.abs(rp) + tol))
        m, v = host(s["avg"][c]), host(s["sq"][c])
        if bits == 32:
            assert np.all(np.abs(m - rm) <= em) and np.all(np.abs(v - rv) <= 16 * H * rv)
            continue
        blocks = slice(c.start // 128, -(-c.stop // 128))
        u = oa.random16(c.stop - c.start, 77, 1, c.start)
        for code, sc, x in ((m, host(s["avg_scale"][blocks]), rm), (v, host(s["sq_scale"][blocks]), np.sqrt(rv))):
            assert np.all(np.abs(sc - oa.moment_scale(x)) <= 16 * H * oa.moment_scale(x))
            want, step = oa.code_steps(x, sc, u)
            near = 16 * 16 * H  # |y| / step is at most 16, off by 16 h of itself: another code only there
            got = np.abs(code) / step
            low, high = np.floor(want - near), np.floor(want + near)
            if x is not rm:
                low, high = np.where(x > 0, np.maximum(low, 1), low), np.where(x > 0, np.maximum(high, 1), high)
            assert np.all((got >= low) & (got <= high)) and np.all((code == 0) | (np.sign(code) == np.sign(x)))
