"""Timed cases of the operators around an adapted layer: 8-bit linear layers and the AdamW step.

  quantize  a matrix to 8-bit floats with one power-of-two scale per 1 x 128 or 128 x 128 block
  forward   y = x W^T with W (and x, quantised in the call) in 8-bit blocks
  backward  dx = dy W, the input gradient of the same frozen layer
  adamw     one AdamW step over all adapters of a model, moments in 32 or 8 bits, optionally with a
            float32 master copy of the weights and clipping by the global gradient norm

`run` computes a case in elementary torch operations, or (own = True) with the package's calls.
Layer sizes are the ones of the package's workloads (c2 ... c5 in dora_inputs).
"""
import math

import torch

own = False

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOAT = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
BETAS, EPS, DECAY, LR = (0.9, 0.999), 1e-8, 0.01, 1e-4
SEED, DONE = 1234, 100  # of the stochastic rounding; steps done before the timed one

# ------------------------------------------------------------------ cases


def listed():
    return [
        # the activations of a 4096-token batch in front of an 8192-wide layer
        dict(name="quantize rows 4096x8192", op="quantize", rows=4096, cols=8192, dtype="bf16", block="row", fp8="e4m3"),
        # a merged up-projection weight on its way into 8 bits
        dict(name="quantize tiles 27648x5120", op="quantize", rows=27648, cols=5120, dtype="bf16", block="tile", fp8="e4m3"),
        # one generated token through an attention projection: latency
        dict(name="forward T1 4096x4096", op="forward", T=1, d_out=4096, d_in=4096, dtype="bf16", fp8="e4m3"),
        # a ragged batch of generated tokens through the widest layer: the weight's bytes
        dict(name="forward T37 27648x5120", op="forward", T=37, d_out=27648, d_in=5120, dtype="bf16", fp8="e4m3"),
        # a short prompt in float32
        dict(name="forward T512 6144x2048 fp32", op="forward", T=512, d_out=6144, d_in=2048, dtype="fp32", fp8="e4m3"),
        # a training batch through a square layer, and the largest product of the workloads
        dict(name="forward T4096 8192x8192", op="forward", T=4096, d_out=8192, d_in=8192, dtype="bf16", fp8="e4m3"),
        dict(name="forward T8192 27648x5120", op="forward", T=8192, d_out=27648, d_in=5120, dtype="bf16", fp8="e4m3"),
        # input gradients: a small batch, and a training batch with the wider-ranged gradient format
        dict(name="backward T512 2048x6144", op="backward", T=512, d_out=2048, d_in=6144, dtype="bf16", fp8="e4m3"),
        dict(name="backward T4096 8192x8192", op="backward", T=4096, d_out=8192, d_in=8192, dtype="bf16", fp8="e5m2"),
        # one adapted layer, float32 moments and master weights, clipped: latency
        dict(name="adamw32 1 layer r64", op="adamw", layers=1, d_out=2048, d_in=6144, r=64, dtype="bf16", bits=32, master=True, clip=True),
        # 384 small tensors: every attention projection of a 32-layer model
        dict(name="adamw8 128 layers r16", op="adamw", layers=128, d_out=4096, d_in=4096, r=16, dtype="bf16", bits=8, master=False, clip=False),
        # a hundred million trained values at a high rank
        dict(name="adamw8 16 layers r384", op="adamw", layers=16, d_out=8192, d_in=8192, r=384, dtype="bf16", bits=8, master=True, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    return max(16, _log(rng, lo, hi) // 16 * 16)  # 8-bit rows are whole 16-byte pieces


def draw(rng):
    op = rng.choice(["quantize", "forward", "forward", "backward", "adamw", "adamw"])
    if op == "quantize":
        cols = _wide(rng, 64, 27648)
        return dict(op=op, rows=_log(rng, 1, min(27648, 27648 * 5120 // cols)), cols=cols, dtype=rng.choice(["bf16", "fp32"]),
                    block=rng.choice(["row", "tile"]), fp8=rng.choice(["e4m3", "e5m2"]))
    if op in ("forward", "backward"):
        d_out, d_in = _wide(rng, 256, 27648), _wide(rng, 256, 27648)
        most = 27648 * 5120
        while d_out * d_in > most:
            d_out, d_in = max(16, d_out // 32 * 16), d_in
        return dict(op=op, T=_log(rng, 1, 8192), d_out=d_out, d_in=d_in, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    fp8="e4m3" if op == "forward" else rng.choice(["e4m3", "e5m2"]))
    r, d_out, d_in = 8 * _log(rng, 1, 48), 8 * _log(rng, 64, 1024), 8 * _log(rng, 64, 1024)
    most = 16 * (384 * 16384 + 8192)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    return dict(op=op, layers=_log(rng, 1, max(1, min(128, most // (r * (d_out + d_in) + d_out)))), d_out=d_out, d_in=d_in, r=r,
                dtype=dtype, bits=rng.choice([8, 8, 32]), master=dtype == "bf16" and rng.choice([True, False]),
                clip=rng.choice([True, False]))


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, cols, dtype):
    """Unit normal with a few wide channels, as hidden states have, and one row of padding."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x[:, torch.randint(0, cols, (max(1, cols // 256),), generator=g, device="cuda")] *= 20.0
    if rows > 4:
        x[rows // 2] = 0.0
    return x.to(FLOAT[dtype])


def _segments(case):
    """Lengths of the trained tensors: all A and B first, then all m."""
    d_out, d_in, r = case["d_out"], case["d_in"], case["r"]
    return [r * d_in, d_out * r] * case["layers"], [d_out] * case["layers"]


def _padded(lengths):
    return [-(-n // 128) * 128 for n in lengths]


def _views(flat, lengths):
    return [v[:n] for v, n in zip(flat.split(_padded(lengths)), lengths)]


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quantize":
        if case["block"] == "row":
            return dict(case=case, x=_activations(g, case["rows"], case["cols"], case["dtype"]))
        w = torch.randn(case["rows"], case["cols"], generator=g, device="cuda") * 0.02
        return dict(case=case, x=w.to(FLOAT[case["dtype"]]))
    if case["op"] in ("forward", "backward"):
        w = torch.randn(case["d_out"], case["d_in"], generator=g, device="cuda") * 0.02
        wq, ws = _quantize_tiles(w, "e4m3")
        if case["op"] == "forward":
            x = _activations(g, case["T"], case["d_in"], case["dtype"])
        else:
            x = (_activations(g, case["T"], case["d_out"], "fp32") * 1e-3).to(FLOAT[case["dtype"]])
        return dict(case=case, x=x, wq=wq, ws=ws)
    mats, vecs = _segments(case)
    nm, nv = sum(_padded(mats)), sum(_padded(vecs))
    n = nm + nv
    pad = torch.zeros(n, dtype=torch.bool, device="cuda")
    if nm + nv != sum(mats) + sum(vecs):  # the padding behind each tensor's last block holds zeros
        pad = torch.cat([(torch.arange(p, device="cuda") >= k) for k, p in zip(mats + vecs, _padded(mats + vecs))])
    size = torch.exp(torch.randn(n // 128, 1, generator=g, device="cuda")).expand(-1, 128).reshape(-1) * 1e-3
    grad = (torch.randn(n, generator=g, device="cuda") * size).masked_fill_(pad, 0.0)
    avg = (torch.randn(n, generator=g, device="cuda") * size * 0.25).masked_fill_(pad, 0.0)
    root = (torch.rand(n, generator=g, device="cuda").add_(0.05) * size).masked_fill_(pad, 0.0)
    param = (torch.randn(n, generator=g, device="cuda") * 0.01).masked_fill_(pad, 0.0)
    param[nm:].add_(1.0).masked_fill_(pad[nm:], 0.0)
    t = FLOAT[case["dtype"]]
    s = dict(case=case, step=DONE, p=param[:nm].to(t), pv=param[nm:].clone(), g=grad[:nm].to(t), gv=grad[nm:].clone())
    if case["master"]:
        s["master"] = s["p"].float()  # of the bf16 tensors; m is float32 already
    if case["bits"] == 32:
        s["avg"], s["sq"] = avg, root.square()
    else:
        s["avg"], s["avg_scale"] = _codes(avg)
        s["sq"], s["sq_scale"] = _codes(root)
    s["decay"] = torch.cat([torch.full((nm,), DECAY, device="cuda"), torch.zeros(nv, device="cuda")])
    if own:  # the handle that a training program keeps, over the same tensors
        import dora_weight_decomposed_b200 as dw

        s["opt"] = dw.DoraAdamW(_views(s["p"], mats) + _views(s["pv"], vecs), _views(s["g"], mats) + _views(s["gv"], vecs),
                                lr=LR, betas=BETAS, eps=EPS, weight_decay=[DECAY] * len(mats) + [0.0] * len(vecs),
                                state_bits=case["bits"], master=case["master"], seed=SEED)
        s["opt"].load_state_dict({k: s[k] for k in ("avg", "sq", "avg_scale", "sq_scale", "master", "step") if k in s})
    return s


# ------------------------------------------------------------------ the plain forms


def _scale(amax, top):
    """2^e with the smallest e that has amax <= top 2^e (top is 1.75 2^k); a non-finite amax is its own scale."""
    mant, ex = torch.frexp(amax)  # amax = mant 2^ex, mant in [0.5, 1)
    e = ex - int(math.log2(top / 1.75)) - 1 + (mant > 0.875).int()
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    scale = ((e + 127) << 23).view(torch.float32)
    return torch.where(torch.isfinite(amax), scale, amax)


def _quantize_rows(x, fp8):
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, 128)
    scale = _scale(v.abs().amax(dim=2), TOP[fp8])
    q = (v / scale[:, :, None]).to(FP8[fp8]).view(rows, -1)[:, :cols].contiguous()
    return q, scale.t().contiguous()


def _quantize_tiles(x, fp8):
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -cols % 128, 0, -rows % 128))
    v = v.view(v.shape[0] // 128, 128, v.shape[1] // 128, 128)
    scale = _scale(v.abs().amax(dim=(1, 3)), TOP[fp8])
    q = (v / scale[:, None, :, None]).view(v.shape[0] * 128, -1)[:rows, :cols].to(FP8[fp8])
    return q.contiguous(), scale


def _dequantize_tiles(q, scale):
    wide = scale.repeat_interleave(128, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, : q.shape[1]]
    return q.float() * wide


def _moment_scale(b):
    """A block's largest moment is held as code 448: the scale follows it without a step."""
    return (b.abs().amax(dim=1) / 448.0).clamp(min=2.0 ** -126)


def _codes(v):
    """8-bit moments rounded to nearest: what earlier steps have left."""
    b = v.view(-1, 128)
    scale = _moment_scale(b)
    return (b / scale[:, None]).to(torch.float8_e4m3fn).view(-1), scale


def _random16(n, step, device):
    """16 random bits for each of n values: an integer hash of (seed, step, index / 2), the low half for even indices."""
    def mix(x):
        x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
        x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
        return x ^ (x >> 16)

    key = mix(torch.tensor((SEED + step * 0x9E3779B9) & 0xFFFFFFFF, device=device))
    h = mix(torch.arange((n + 1) // 2, device=device) ^ key)
    return torch.stack([h & 0xFFFF, h >> 16], dim=1).view(-1)[:n]


def _store_codes(v, u):
    """v as 8-bit codes: scaled by block, then floor(y / step + u) steps, step being the code's spacing at y."""
    b = v.view(-1, 128)
    scale = _moment_scale(b)
    y = b / scale[:, None]
    low = y.abs() < 2.0 ** -6  # below the normal codes the spacing stays 2^-9
    a = y.abs() + torch.where(low, 2.0 ** -6, 0.0)
    bits = ((a.view(torch.int32) + (u.view(-1, 128).int() << 4)) >> 20) << 20
    a = bits.view(torch.float32) - torch.where(low, 2.0 ** -6, 0.0)
    return torch.copysign(a, y), scale


def _adamw(s):
    case = s["case"]
    s["step"] += 1
    t, (b1, b2) = s["step"], BETAS
    nm = s["p"].numel()
    grad = torch.cat([s["g"].float(), s["gv"]])
    out = {}
    if case["clip"]:
        norm = grad.double().square().sum().sqrt()
        grad = grad * torch.clamp(1.0 / (norm + 1e-6), max=1.0).float()
        out["norm"] = norm.float()
    param = torch.cat([s["master"] if case["master"] else s["p"].float(), s["pv"]])
    if case["bits"] == 32:
        avg, sq = s["avg"], s["sq"]
    else:
        avg = (s["avg"].float().view(-1, 128) * s["avg_scale"][:, None]).view(-1)
        sq = (s["sq"].float().view(-1, 128) * s["sq_scale"][:, None]).square().view(-1)
    avg = avg * b1 + grad * (1 - b1)
    sq = sq * b2 + grad * grad * (1 - b2)
    root = sq.sqrt()
    param = param - param * s["decay"] * LR - (avg * (LR / (1 - b1 ** t))) / (root * (1 / math.sqrt(1 - b2 ** t)) + EPS)
    if case["bits"] == 32:
        s["avg"], s["sq"] = avg, sq
    else:
        u = _random16(avg.numel(), t, avg.device)
        code, s["avg_scale"] = _store_codes(avg, u)
        s["avg"] = code.to(torch.float8_e4m3fn).view(-1)
        code, s["sq_scale"] = _store_codes(root, u)
        code = torch.where((code == 0) & (root.view(-1, 128) > 0), 2.0 ** -9, code)  # a nonzero moment is never held as zero
        s["sq"] = code.to(torch.float8_e4m3fn).view(-1)
    s["p"], s["pv"] = param[:nm].to(s["p"].dtype), param[nm:].clone()
    if case["master"]:
        s["master"] = param[:nm].clone()
    return {**out, **{k: s[k] for k in ("p", "pv", "avg", "sq", "avg_scale", "sq_scale", "master") if k in s}}


def run(state):
    case = state["case"]
    if own:
        import dora_weight_decomposed_b200 as dw

        if case["op"] == "quantize":
            return dw.dora_fp8_quantize(state["x"], block=case["block"], dtype=FP8[case["fp8"]])
        if case["op"] == "forward":
            return dw.dora_fp8_forward(state["x"], state["wq"], state["ws"], fp8_dtype=FP8[case["fp8"]])
        if case["op"] == "backward":
            return dw.dora_fp8_backward(state["x"], state["wq"], state["ws"], fp8_dtype=FP8[case["fp8"]])
        opt = state["opt"]
        norm = opt.step(max_norm=1.0 if case["clip"] else None)
        out = {"norm": norm} if case["clip"] else {}
        return {**out, "p": state["p"], "pv": state["pv"], **{k: v for k, v in opt.state_dict().items() if k != "step"}}
    if case["op"] == "quantize":
        return (_quantize_rows if case["block"] == "row" else _quantize_tiles)(state["x"], case["fp8"])
    if case["op"] == "adamw":
        return _adamw(state)
    q, scale = _quantize_rows(state["x"], case["fp8"])
    x = q.float() * scale.t().repeat_interleave(128, 1)[:, : q.shape[1]]
    w = _dequantize_tiles(state["wq"], state["ws"])
    return torch.matmul(x, w.t() if case["op"] == "forward" else w).to(state["x"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        up = -(-case["cols"] // 128) * (case["rows"] if case["block"] == "row" else -(-case["rows"] // 128))
        return {"bytes": n * (BYTES[case["dtype"]] + 1) + 4 * up, "flops": 2 * n}
    if case["op"] in ("forward", "backward"):
        T, d_out, d_in = case["T"], case["d_out"], case["d_in"]
        tiles = -(-d_out // 128) * -(-d_in // 128)
        return {"bytes": BYTES[case["dtype"]] * T * (d_in + d_out) + d_out * d_in + 4 * tiles, "flops": 2 * T * d_out * d_in}
    mats, vecs = _segments(case)
    n = sum(mats) + sum(vecs)
    b = BYTES[case["dtype"]]
    moments = n * (16 if case["bits"] == 32 else 4 + 16 / 128)
    weights = sum(mats) * (b + 8 if case["master"] else 2 * b) + sum(vecs) * 8
    return {"bytes": sum(mats) * b + sum(vecs) * 4 + weights + moments, "flops": 20 * n}


# ------------------------------------------------------------------ 64 bits, from the definitions


def _power64(e):
    """2^e exactly (pow() may be a unit off, and a tie is then no tie)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _code64(y, fp8, u=None):
    """The 8-bit value next to y (ties to even), or with u in [0, 1): floor(|y| / step + u) steps."""
    low, mant = (-6, 3) if fp8 == "e4m3" else (-14, 2)
    _, ex = torch.frexp(y)
    step = _power64((ex - 1).clamp(min=low) - mant)
    a = torch.round(y / step) if u is None else torch.floor(y.abs() / step + u) * torch.sign(y)
    return (a * step).clamp(-TOP[fp8], TOP[fp8])


def _scale64(amax, fp8):
    e = torch.ceil(torch.log2(amax / TOP[fp8]) - 1e-12).clamp(min=-126)  # amax has 24 bits: no value is that near a border
    return _power64(e)


def _blocks64(x, fp8, tile):
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 128, 0, -rows % 128 if tile else 0))
    v = v.unflatten(1, (-1, 128))
    if tile:
        v = v.unflatten(0, (-1, 128))
        s = _scale64(v.abs().amax(dim=(1, 3), keepdim=True), fp8)
        return _code64(v / s, fp8).flatten(2).flatten(0, 1)[:rows, :cols], s[:, 0, :, 0]
    s = _scale64(v.abs().amax(dim=2, keepdim=True), fp8)
    return _code64(v / s, fp8).flatten(1)[:, :cols], s[:, :, 0]


def _exact_adamw(s):
    case, (b1, b2), t = s["case"], BETAS, s["step"] + 1
    nm = s["p"].numel()
    g = torch.cat([s["g"].double(), s["gv"].double()])
    norm = torch.linalg.vector_norm(g)
    if case["clip"] and norm + 1e-6 > 1.0:
        g = g / (norm + 1e-6)
    p = torch.cat([s["master" if case["master"] else "p"].double(), s["pv"].double()])
    m, v = s["avg"].double(), s["sq"].double()
    if case["bits"] == 8:
        m = m * s["avg_scale"].double().repeat_interleave(128)
        v = (v * s["sq_scale"].double().repeat_interleave(128)) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - LR * s["decay"].double()) - LR * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + EPS)
    out = {"p": p[:nm], "pv": p[nm:], "avg": m, "sq": v}
    if case["clip"]:
        out["norm"] = norm
    if case["master"]:
        out["master"] = p[:nm]
    if case["bits"] == 8:
        u = _random16(m.numel(), t, m.device).double().view(-1, 128) / 65536  # the random numbers are inputs
        m, r = m.view(-1, 128), v.sqrt().view(-1, 128)
        ms, rs = ((x.abs().amax(dim=1, keepdim=True) / 448.0).clamp(min=2.0 ** -126) for x in (m, r))
        r8 = _code64(r / rs, "e4m3", u)
        out["avg"], out["avg_scale"] = _code64(m / ms, "e4m3", u).flatten(), ms.flatten()
        out["sq"], out["sq_scale"] = torch.where(r > 0, r8.clamp(min=2.0 ** -9), r8).flatten(), rs.flatten()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] == "quantize":
        q, scale = _blocks64(s["x"], case["fp8"], case["block"] == "tile")
        return q, (scale if case["block"] == "tile" else scale.t())
    q, scale = _blocks64(s["x"], case["fp8"], False)
    x = q * scale.repeat_interleave(128, 1)[:, : q.shape[1]]
    w = s["wq"].double() * s["ws"].double().repeat_interleave(128, 0)[: case["d_out"]].repeat_interleave(128, 1)[:, : case["d_in"]]
    return x @ (w.t() if case["op"] == "forward" else w)
