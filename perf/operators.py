"""Cases, plain forms and exact values of the block-FP8 feed-forward operators.

rms     rmsnorm_residual_quant_fp8: h = bf16(x + residual), RMS norm, E4M3 codes with one scale per 128 or per row
quant   quant_act_fp8_per128: BF16 activations -> E4M3 codes with one scale per 128
silu    silu_mul_quant_fp8_per128: silu(gate) * up -> E4M3 codes with one scale per 128
gemm    fp8_gemm_blockscaled: 1x128-scaled activations x 128x128-scaled weight -> BF16
moe     fp8_moe_blockscaled: router choice, gate/up, SiLU, down and combination for at most 16 tokens

`run` computes the plain forms in 32 bits, or calls the library where `own` is
true.  E4M3 codes are returned as torch.float8_e4m3fn, the values they stand for.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # the norm in front of a projection: one decoded token; a ragged batch feeding the row-scaled GEMM, first
        # layer (no residual); a long prefill
        {"name": "rms_token", "op": "rms", "m": 1, "k": 5120, "group": 128, "residual": True},
        {"name": "rms_ragged_rows", "op": "rms", "m": 777, "k": 4112, "group": 0, "residual": False},
        {"name": "rms_prefill", "op": "rms", "m": 8192, "k": 5120, "group": 128, "residual": True},
        # activations that no norm produces (attention output): a decode batch; a prefill at the widest K
        {"name": "quant_decode", "op": "quant", "m": 16, "k": 5120},
        {"name": "quant_prefill", "op": "quant", "m": 4096, "k": 17408},
        # between the two products of a gated MLP: a small decode batch; a prefill
        {"name": "silu_decode", "op": "silu", "m": 5, "k": 17408},
        {"name": "silu_prefill", "op": "silu", "m": 2048, "k": 17408},
        # projections: a decode batch (the weight stream); ragged rows and an N that ends inside a scale block; the
        # benchmark's large prefill
        {"name": "gemm_decode", "op": "gemm", "m": 16, "n": 5120, "k": 5120},
        {"name": "gemm_ragged", "op": "gemm", "m": 777, "n": 2112, "k": 5120},
        {"name": "gemm_prefill", "op": "gemm", "m": 4096, "n": 17408, "k": 5120},
        # expert layers: one decoded token; a full decode batch that touches nearly every expert
        {"name": "moe_token", "op": "moe", "t": 1, "h": 2048, "i": 768, "e": 64, "topk": 8, "masked": 0, "renorm": True},
        {"name": "moe_batch", "op": "moe", "t": 16, "h": 5120, "i": 1408, "e": 64, "topk": 8, "masked": 3,
         "renorm": False},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["rms", "quant", "silu", "gemm", "gemm", "moe", "moe"])
    if op == "rms":
        group = rng.choice([0, 128])
        return {"op": op, "m": _log(rng, 1, 8192), "k": _log(rng, 256, 5120, 128 if group else 16), "group": group,
                "residual": rng.random() < 0.7}
    if op == "quant":
        return {"op": op, "m": _log(rng, 1, 4096), "k": _log(rng, 128, 17408, 128)}
    if op == "silu":
        return {"op": op, "m": _log(rng, 1, 2048), "k": _log(rng, 128, 17408, 128)}
    if op == "gemm":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 64, 17408, rng.choice([1, 8, 128])),
                "k": _log(rng, 256, 5120, 128)}
    e = _log(rng, 8, 64)
    topk = rng.randint(1, min(8, e // 2))
    return {"op": op, "t": rng.randint(1, 16), "h": _log(rng, 1024, 5120, 128), "i": _log(rng, 384, 1408, 128),
            "e": e, "topk": topk, "masked": rng.randint(0, e // 4), "renorm": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs ---

def _activations(g, m, k):
    """BF16 activations with a few channels far above the others, as hidden states have."""
    x = torch.randn(m, k, device=DEV, generator=g)
    x *= 1.0 + 19.0 * (torch.rand(k, device=DEV, generator=g) < 0.01)
    return x.bfloat16()


def _row_codes(x):
    """Activations as E4M3 codes with one scale per 128 (what the quantiser in front of the product leaves)."""
    m, k = x.shape
    v = x.float().view(m, k // 128, 128)
    s = v.abs().amax(-1) / 448.0
    q = (v / torch.where(s == 0, 1.0, s)[..., None]).clamp(-448, 448).to(F8)
    return q.view(m, k).view(torch.uint8), s


def _weight(g, n, k, experts=None):
    """A weight ~ N(0, 0.02) as E4M3 codes with one scale per 128 x 128 block (the last row block may be short)."""
    e, nb = experts or 1, -(-n // 128)
    w = torch.randn(e, nb * 128, k, device=DEV, generator=g).mul_(0.02)
    b = w.view(e, nb, 128, k // 128, 128)
    s = b.abs().amax(dim=(2, 4)) / 448.0
    q = (b / s[:, :, None, :, None]).clamp(-448, 448).to(F8).view(torch.uint8).view(e, nb * 128, k)[:, :n].contiguous()
    return (q, s) if experts else (q[0], s[0])


def _empty(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    if c["op"] == "moe":
        t, h, i, e = c["t"], c["h"], c["i"], c["e"]
        c["x"] = _activations(g, t, h)
        c["logits"] = torch.randn(t, e, device=DEV, generator=g)
        if c["masked"]:  # experts that this group of tokens may not use
            c["logits"][:, torch.randperm(e, device=DEV, generator=g)[:c["masked"]]] = -math.inf
        c["w13"], c["s13"] = _weight(g, 2 * i, h, e)
        c["w2"], c["s2"] = _weight(g, h, i, e)
        c["out"] = _empty(t, h, dtype=torch.bfloat16)
        c["ids"] = _empty(t, c["topk"], dtype=torch.int32)
        c["tw"] = _empty(t, c["topk"], dtype=torch.float32)
        return c
    m, k = c["m"], c["k"]
    if c["op"] == "gemm":
        c["a"], c["sa"] = _row_codes(_activations(g, m, k))
        c["w"], c["sw"] = _weight(g, c["n"], k)
        c["out"] = _empty(m, c["n"], dtype=torch.bfloat16)
        return c
    c["x"] = _activations(g, m, 2 * k if c["op"] == "silu" else k)
    c["q"] = _empty(m, k, dtype=torch.uint8)
    c["s"] = _empty(m, k // 128, dtype=torch.float32)
    if c["op"] == "rms":
        c["gain"] = (1.0 + 0.2 * torch.randn(k, device=DEV, generator=g)).bfloat16()
        if c["group"] == 0:
            c["s"] = _empty(m, dtype=torch.float32)
        c["res"] = _activations(g, m, k) if c["residual"] else None
        c["res_out"] = _empty(m, k, dtype=torch.bfloat16) if c["residual"] else None
    return c


# ------------------------------------------------------------ plain forms ---

def _codes(y, group):
    """FP32 rows -> E4M3 codes of y / s, s = amax / 448 over each group (0: the whole row)."""
    m, k = y.shape
    v = y.view(m, k // (group or k), group or k)
    s = v.abs().amax(-1) / 448.0
    q = (v / torch.where(s == 0, 1.0, s)[..., None]).clamp(-448.0, 448.0).to(F8).view(m, k)
    return q, (s if group else s[:, 0])


def _plain_rms(c):
    h = c["x"].float()
    if c["residual"]:
        h = (h + c["res"].float()).bfloat16().float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * c["gain"].float()
    q, s = _codes(y, c["group"])
    return {"q": q, "s": s, "h": h.bfloat16()} if c["residual"] else {"q": q, "s": s}


def _plain_silu(c):
    gate, up = c["x"].float().split(c["k"], dim=1)
    q, s = _codes(gate / (1.0 + torch.exp(-gate)) * up, 128)
    return {"q": q, "s": s}


def _dequant(w, s):
    """E4M3 codes [..., n, k] x one scale per 128 x 128 block -> FP32."""
    n = w.shape[-2]
    rows = s.repeat_interleave(128, dim=-2)[..., :n, :]
    return (w.view(F8).float().unflatten(-1, (-1, 128)) * rows[..., None]).flatten(-2)


def _plain_gemm(c):
    a = (c["a"].view(F8).float().unflatten(-1, (-1, 128)) * c["sa"][..., None]).flatten(-2)
    return {"out": (a @ _dequant(c["w"], c["sw"]).t()).bfloat16()}


def _plain_moe(c):
    t, i, e, topk = c["t"], c["i"], c["e"], c["topk"]
    x, logits = c["x"].float(), c["logits"]
    top, order = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: the lowest index first
    ids = order[:, :topk]
    p = torch.exp(logits - top[:, :1])
    pk = torch.gather(p, 1, ids)
    tw = pk / (pk if c["renorm"] else p).sum(-1, keepdim=True)
    if t * topk < e:  # the chosen experts' weights, one (token, expert) pair each
        sel = ids.reshape(-1)
        gu = _dequant(c["w13"][sel], c["s13"][sel]) @ x.repeat_interleave(topk, 0)[:, :, None]  # [pairs, 2i, 1]
        gate, up = gu[:, :i], gu[:, i:]
        y = _dequant(c["w2"][sel], c["s2"][sel]) @ (gate / (1.0 + torch.exp(-gate)) * up)  # [pairs, h, 1]
        out = (y.view(t, topk, -1) * tw[..., None]).sum(1)
    else:  # every expert for every token, weighted by the token's choice
        gu = _dequant(c["w13"], c["s13"]) @ x.t()  # [e, 2i, t]
        gate, up = gu[:, :i], gu[:, i:]
        y = _dequant(c["w2"], c["s2"]) @ (gate / (1.0 + torch.exp(-gate)) * up)  # [e, h, t]
        dense = torch.zeros_like(logits).scatter_(1, ids, tw)  # [t, e]
        out = (y * dense.t()[:, None, :]).sum(0).t()
    return {"out": out.bfloat16(), "ids": ids.int(), "tw": tw}


# ---------------------------------------------------------- library calls ---

def _own(c):
    import int8_gemm_gemv_b200 as bsq

    op = c["op"]
    if op == "rms":
        bsq.rmsnorm_residual_quant_fp8(c["x"], c["res"], c["gain"], EPS, c["res_out"], c["q"], c["s"], c["group"],
                                       c["m"], c["k"])
        out = {"q": c["q"].view(F8), "s": c["s"]}
        return dict(out, h=c["res_out"]) if c["residual"] else out
    if op == "quant":
        bsq.quant_act_fp8_per128(c["x"], c["q"], c["s"], c["m"], c["k"])
        return {"q": c["q"].view(F8), "s": c["s"]}
    if op == "silu":
        bsq.silu_mul_quant_fp8_per128(c["x"], c["q"], c["s"], c["m"], c["k"])
        return {"q": c["q"].view(F8), "s": c["s"]}
    if op == "gemm":
        bsq.fp8_gemm_blockscaled(c["a"], c["sa"], c["w"], c["sw"], c["out"], c["m"], c["n"], c["k"])
        return {"out": c["out"]}
    if "ws" not in c:  # the workspace a serving loop keeps
        c["ws_bytes"] = bsq.fp8_moe_workspace_bytes(c["t"], c["h"], c["i"], c["topk"])
        c["ws"] = _empty(c["ws_bytes"], dtype=torch.uint8)
    bsq.fp8_moe_blockscaled(c["x"], c["logits"], c["w13"], c["s13"], c["w2"], c["s2"], c["out"], c["ids"], c["tw"],
                            c["ws"], c["ws_bytes"], c["t"], c["h"], c["i"], c["e"], c["topk"], c["renorm"])
    return {"out": c["out"], "ids": c["ids"], "tw": c["tw"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "rms":
        return _plain_rms(state)
    if op == "quant":
        q, s = _codes(state["x"].float(), 128)
        return {"q": q, "s": s}
    if op == "silu":
        return _plain_silu(state)
    return _plain_gemm(state) if op == "gemm" else _plain_moe(state)


# ------------------------------------------------------------------- work ---

def work(case):
    c = case
    if c["op"] == "moe":
        t, h, i, e, topk = c["t"], c["h"], c["i"], c["e"], c["topk"]
        usable = e - c["masked"]
        hit = usable * (1.0 - (1.0 - topk / usable) ** t)  # experts that t tokens reach, on average
        weights = hit * (3 * h * i + 4 * 3 * (h // 128) * (i // 128))
        return {"bytes": weights + 4 * t * h + 4 * t * e + 8 * t * topk, "flops": 6.0 * t * topk * h * i}
    m, k = c["m"], c["k"]
    if c["op"] == "gemm":
        n = c["n"]
        nb = -(-n // 128)
        return {"bytes": m * k + n * k + 4 * (m + nb) * (k // 128) + 2 * m * n, "flops": 2.0 * m * n * k}
    codes = m * k + 4 * m * (k // 128)
    if c["op"] == "rms":
        scales = 4 * m * (k // c["group"] if c["group"] else 1)
        return {"bytes": m * k * (6 if c["residual"] else 2) + 2 * k + m * k + scales, "flops": 6.0 * m * k}
    if c["op"] == "quant":
        return {"bytes": 2 * m * k + codes, "flops": 2.0 * m * k}
    return {"bytes": 4 * m * k + codes, "flops": 7.0 * m * k}


# ------------------------------------------------------------------ exact ---

def _nearest_e4m3(x):
    """The E4M3 value nearest each FP64 value (ties to even, saturating at 448)."""
    a = x.abs()
    _, ex = torch.frexp(a)  # a = f * 2^ex, f in [1/2, 1)
    step = torch.ldexp(torch.ones_like(a), (ex - 1).clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def _exact_codes(y, width):
    m, k = y.shape
    blocks = y.reshape(m * k // width, width)
    s = blocks.abs().max(dim=1, keepdim=True).values / 448.0
    return {"q": _nearest_e4m3(torch.where(s > 0, blocks / s, torch.zeros_like(blocks))).reshape(m, k),
            "s": s.reshape(m, k // width)}


def _exact_weight(w, s):
    out = w.view(F8).double()
    r = torch.arange(w.shape[-2], device=DEV) // 128
    col = torch.arange(w.shape[-1], device=DEV) // 128
    return out * s.double()[..., r, :][..., col]


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op == "quant":
        return _exact_codes(c["x"].double(), 128)
    if op == "silu":
        x = c["x"].double()
        return _exact_codes(x[:, :c["k"]] * torch.sigmoid(x[:, :c["k"]]) * x[:, c["k"]:], 128)
    if op == "rms":
        h = c["x"].double()
        if c["residual"]:
            h = (h + c["res"].double()).bfloat16().double()
        y = h * c["gain"].double() / torch.sqrt((h ** 2).sum(1, keepdim=True) / c["k"] + EPS)
        r = _exact_codes(y, c["group"] or c["k"])
        if c["group"] == 0:
            r["s"] = r["s"].reshape(c["m"])
        return dict(r, h=h) if c["residual"] else r
    if op == "gemm":
        col = torch.arange(c["k"], device=DEV) // 128
        return {"out": (c["a"].view(F8).double() * c["sa"].double()[:, col]) @ _exact_weight(c["w"], c["sw"]).t()}
    # one expert at a time, for the tokens that chose it
    t, i, topk = c["t"], c["i"], c["topk"]
    logits, x = c["logits"].double(), c["x"].double()
    p = torch.softmax(logits, dim=1)
    ids = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :topk]
    tw = p.gather(1, ids)
    if c["renorm"]:
        tw = tw / tw.sum(1, keepdim=True)
    out = torch.zeros(t, c["h"], dtype=torch.float64, device=DEV)
    for ex in range(c["e"]):
        tok, slot = torch.where(ids == ex)
        if tok.numel():
            gu = x[tok] @ _exact_weight(c["w13"][ex], c["s13"][ex]).t()
            act = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
            out.index_add_(0, tok, tw[tok, slot][:, None] * (act @ _exact_weight(c["w2"][ex], c["s2"][ex]).t()))
    return {"out": out, "ids": ids.int(), "tw": tw}
