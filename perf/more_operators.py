"""Workloads of the operators around an attention: products with 4-bit weights, residual addition with RMSNorm,
rotary positions, and the verification of drafted tokens.

  product  y = W x for a few rows x, W in 4-bit codes: groups of consecutive inputs share a scale d and a zero z, and
           the code n stands for (n - z) d (z = 8 without zeros). x is f32, bf16 or e4m3 codes with scales; a residual
           may be added, and two matrices W and U may be joined to silu(W x) * (U x)
  norm     s = x + residual; y = s / sqrt(mean(s^2) + eps) * gain, as f32, bf16, or e4m3 codes whose blocks share the
           scale max|y| / 448
  rotate   pairs (a, b) of a head's dims at position p become (a cos - b sin, a sin + b cos) of the angle p f, for
           halves or neighbours as pairs, all of the head or its first dims, plain or scaled frequencies f
  verify   drafted tokens x_0, x_1, ... of target distributions p_i and draft distributions q_i: x_i is taken while
           u_i q_i(x_i) < p_i(x_i); the next token is drawn from max(p_i - q_i, 0) where one is refused, else from the
           row after the last

`run` computes the plain form, or with `own` the framework's calls.
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases

def listed():
    def product(name, rows, n, k, group, x, out, zeros, residual, gated):
        return dict(name=name, kind="product", rows=rows, n=n, k=k, group=group, x=x, out=out, zeros=zeros,
                    residual=residual, gated=gated)

    def norm(name, rows, width, x, residual, out, block):
        return dict(name=name, kind="norm", rows=rows, width=width, x=x, residual=residual, out=out, block=block)

    def rotate(name, streams, rows, q_heads, kv_heads, head_dim, rotary, interleaved, scaling, x, far):
        return dict(name=name, kind="rotate", streams=streams, rows=rows, q_heads=q_heads, kv_heads=kv_heads,
                    head_dim=head_dim, rotary=rotary, interleaved=interleaved, scaling=scaling, x=x, far=far)

    def verify(name, seqs, drafts, vocab, x, draft, greedy, ragged):
        return dict(name=name, kind="verify", seqs=seqs, drafts=drafts, vocab=vocab, x=x, draft=draft, greedy=greedy,
                    ragged=ragged)

    return [
        # the Talker's fused q/k/v projection of a single token: latency
        product("product-qkv", 1, 4096, 1024, 32, "f32", "f32", False, False, False),
        # a small batch over sizes that no tile divides
        product("product-odd", 5, 5003, 2087, 64, "bf16", "bf16", False, True, False),
        # gate and up projections of sixteen streams, weights with zero points
        product("product-gated", 16, 13824, 5120, 128, "bf16", "bf16", True, False, True),
        # one token of a wide layer, its row in 8 bits from the norm before it, added to the residual stream
        product("product-wide", 1, 24576, 8192, 128, "e4m3", "f32", False, True, False),
        # one token's residual stream between two blocks of a layer
        norm("norm-row", 1, 1024, "f32", "f32", "f32", 0),
        # a prompt's rows, to 8 bits for the next product
        norm("norm-prompt", 4096, 5120, "bf16", "f32", "e4m3", 128),
        # one token's heads
        rotate("rotate-row", 1, 1, 16, 8, 128, 128, False, "none", "f32", 40000),
        # prompts of several streams at far positions, part of each head, scaled frequencies
        rotate("rotate-prompts", 3, 5001, 32, 8, 128, 64, True, "yarn", "bf16", 120000),
        # few drafts over a codec vocabulary: latency
        verify("verify-codec", 1, 3, 2048, "f32", True, False, False),
        # drafts that come without probabilities (looked up in the prompt), some sequences greedy
        verify("verify-lookup", 7, 10, 32001, "bf16", False, True, True),
        # a batch over a text vocabulary
        verify("verify-batch", 24, 5, 100003, "f32", True, False, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["product", "product", "norm", "rotate", "verify", "verify"])
    if kind == "product":
        rows, gated = _log(rng, 1, 64), rng.random() < 0.3
        most = 24576 * 8192 // (2 if gated else 1) // (1 + rows // 8)
        n = _log(rng, 64, 24576 if most > 24576 * 64 else most // 64)
        return dict(kind=kind, rows=rows, n=n, k=_log(rng, 64, max(64, min(16384, most // n))),
                    group=rng.choice([32, 64, 128]), x=rng.choice(["f32", "bf16", "e4m3"]),
                    out=rng.choice(["f32", "bf16"]), zeros=rng.random() < 0.4,
                    residual=not gated and rng.random() < 0.5, gated=gated)
    if kind == "norm":
        width = _log(rng, 32, 16384)
        return dict(kind=kind, rows=_log(rng, 1, max(1, 4096 * 5120 // width)), width=width,
                    x=rng.choice(["f32", "bf16"]), residual=rng.choice(["none", "f32", "bf16"]),
                    out=rng.choice(["f32", "bf16", "e4m3"]), block=rng.choice([32, 64, 128]))
    if kind == "rotate":
        hd, streams, qh, kvh = rng.choice([32, 64, 80, 128, 256]), rng.randint(1, 8), rng.randint(1, 32), rng.randint(1, 8)
        most = max(1, 3 * 5001 * 40 * 128 // (streams * (qh + kvh) * hd))
        return dict(kind=kind, streams=streams, rows=_log(rng, 1, min(8192, most)), q_heads=qh, kv_heads=kvh,
                    head_dim=hd, rotary=rng.choice([hd, hd // 2]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "smooth"]), x=rng.choice(["f32", "bf16"]),
                    far=_log(rng, 1, 500000))
    seqs, drafts = _log(rng, 1, 32), rng.randint(1, 10)
    most = max(256, min(150000, 24 * 11 * 100003 // (seqs * (2 * drafts + 1))))
    return dict(kind=kind, seqs=seqs, drafts=drafts, vocab=_log(rng, 256, most), x=rng.choice(["f32", "bf16"]),
                draft=rng.random() < 0.6, greedy=rng.random() < 0.4, ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ prepare

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=F32)


def _matrix(g, n, k, group, zeros):
    """Codes [n, ceil(k / 2)] (the even input in the low four bits), scales [n, groups] fp16, zeros [n, groups] or None:
    what a quantizer of N(0, 0.02) weights stores."""
    groups = -(-k // group)
    codes = torch.randint(0, 256, (n, -(-k // 2)), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.006 * (0.75 + 0.5 * _uniform(g, n, groups))).to(torch.float16)
    z = torch.randint(5, 11, (n, groups), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales, z


SCALINGS = {
    "none": None,
    "linear": {"type": "linear", "factor": 4.0},
    "ntk": {"type": "ntk", "factor": 4.0},
    "yarn": {"type": "yarn", "factor": 4.0, "original": 32768, "beta_fast": 32.0, "beta_slow": 1.0},
    "smooth": {"type": "smooth", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0},
}
THETA = 1e6


def prepare(case, seed):
    g = _gen(seed, 1)
    s = {"kind": case["kind"], "case": case}
    if case["kind"] == "product":
        rows, n, k, group = case["rows"], case["n"], case["k"], case["group"]
        s["w"] = [_matrix(g, n, k, group, case["zeros"]) for _ in range(2 if case["gated"] else 1)]
        x = _normal(g, rows, k)
        if case["x"] == "e4m3":
            s["x"], s["xs"] = _to8(x, 128)
        else:
            s["x"], s["xs"] = x.to(DTYPES[case["x"]]), None
        s["res"] = _normal(g, rows, n).to(DTYPES[case["out"]]) if case["residual"] else None
        if own:
            from kv_cached_qwen3_gb300.w4 import W4Matrix
            s["own"] = W4Matrix.pack(*s["w"][0], k=k, group=group, gated_with=s["w"][1] if case["gated"] else None)
    elif case["kind"] == "norm":
        rows, width = case["rows"], case["width"]
        s["x"] = _normal(g, rows, width).to(DTYPES[case["x"]])
        # a residual stream: larger than what is added to it, a few of its dims much larger
        big = torch.where(_uniform(g, width) < 0.01, 20.0, 1.0)
        s["res"] = (3.0 * big * _normal(g, rows, width)).to(DTYPES[case["residual"]]) if case["residual"] != "none" else None
        s["gain"] = 1.0 + 0.05 * _normal(g, width)
    elif case["kind"] == "rotate":
        B, T, D = case["streams"], case["rows"], case["head_dim"]
        # heads as one projection gives them: q, k (and v) of a row behind one another
        heads = case["q_heads"] + 2 * case["kv_heads"]
        qkv = _normal(g, B, T, heads, D).to(DTYPES[case["x"]])
        s["q"], s["k"] = qkv[:, :, :case["q_heads"]], qkv[:, :, case["q_heads"]:case["q_heads"] + case["kv_heads"]]
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["pos"] = start + torch.arange(T, device="cuda", dtype=torch.int32)
        if own:
            from kv_cached_qwen3_gb300.rotary import Rotary
            s["own"] = Rotary(D, rotary_dim=case["rotary"], theta=THETA, interleaved=case["interleaved"],
                              scaling=SCALINGS[case["scaling"]])
    else:
        S, K, V = case["seqs"], case["drafts"], case["vocab"]
        # what output heads give; the draft model's are near the target's
        t = 2.5 * _normal(g, S, K + 1, V)
        d = t[:, :K] + 0.7 * _normal(g, S, K, V)
        s["target"] = t.to(DTYPES[case["x"]])
        s["draft"] = d.to(DTYPES[case["x"]]) if case["draft"] else None
        s["temp"] = 0.6 + 0.5 * _uniform(g, S)
        if case["greedy"]:
            s["temp"][::2] = 0.0
        # drafts drawn from the draft's distribution; without one, what the target finds likely, now and then
        e = -torch.log(_uniform(g, S, K, V).clamp(min=1e-30))
        s["tokens"] = ((d / s["temp"].clamp(min=0.05)[:, None, None]) - torch.log(e)).argmax(-1).to(torch.int32)
        s["count"] = None
        if case["ragged"]:
            s["count"] = torch.randint(0, K + 1, (S,), generator=g, device="cuda", dtype=torch.int32)
        s["u"] = _uniform(g, S, K + 1)
    return s


# ------------------------------------------------------------------ the plain forms

def _to8(y, block):
    """y [rows, width] -> e4m3 codes, and the scales of blocks of a row (0: the row is one block), f32."""
    rows, width = y.shape
    block = block or width
    b = torch.nn.functional.pad(y, (0, -width % block)).unflatten(-1, (-1, block))
    top = b.abs().amax(-1)
    inv = torch.where(top > 0, 448.0 / top, 0.0)
    codes = (b * inv[..., None]).clamp(-448.0, 448.0).flatten(1)[:, :width].to(torch.float8_e4m3fn)
    return codes, top / 448.0


def _values(x, xs):
    """Rows of f32, bf16, or e4m3 with the scales of blocks of 128, as f32."""
    x = x.to(F32)
    return x if xs is None else x * xs.repeat_interleave(128, -1)[:, :x.shape[1]]


def _dense(w, k, group):
    codes, scales, zeros = w
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :k].to(F32)
    z = 8.0 if zeros is None else zeros.to(F32).repeat_interleave(group, -1)[:, :k]
    return (n - z) * scales.to(F32).repeat_interleave(group, -1)[:, :k]


def _product(s):
    c = s["case"]
    if own:
        return s["own"].matmul(s["x"], x_scales=s["xs"], residual=s["res"], out_dtype=DTYPES[c["out"]])
    x = _values(s["x"], s["xs"])
    y = x @ _dense(s["w"][0], c["k"], c["group"]).T
    if c["gated"]:
        y = y / (1.0 + torch.exp(-y)) * (x @ _dense(s["w"][1], c["k"], c["group"]).T)
    if s["res"] is not None:
        y = y + s["res"].to(F32)
    return y.to(DTYPES[c["out"]])


EPS = 1e-6


def _norm(s):
    c = s["case"]
    if own:
        from kv_cached_qwen3_gb300.norm import rms_norm
        got = rms_norm(s["x"], s["gain"], eps=EPS, residual=s["res"], out_dtype=DTYPES[c["out"]], block=c["block"])
        return dict(zip(("y", "sum", "scales"), got))
    t = s["x"].to(F32)
    total = None
    if s["res"] is not None:
        t = t + s["res"].to(F32)
        total = t.to(s["res"].dtype)
    y = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS) * s["gain"]
    if c["out"] == "e4m3":
        codes, scales = _to8(y, c["block"])
        return {"y": codes, "sum": total, "scales": scales}
    return {"y": y.to(DTYPES[c["out"]]), "sum": total, "scales": None}


def _frequencies(rotary, scaling):
    """Radians a position, [rotary / 2] in 64 bits, and the factor of cos and sin."""
    c = SCALINGS[scaling]
    i = torch.arange(rotary // 2, dtype=F64, device="cuda")
    f = THETA ** (-2.0 * i / rotary)
    if c is None:
        return f, 1.0
    if c["type"] == "linear":
        return f / c["factor"], 1.0
    if c["type"] == "ntk":
        return (THETA * c["factor"] ** (rotary / (rotary - 2.0))) ** (-2.0 * i / rotary), 1.0
    turns = c["original"] * f / (2.0 * math.pi)               # turns over the original context
    if c["type"] == "smooth":
        keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0.0, 1.0)
        return f * keep + f / c["factor"] * (1.0 - keep), 1.0
    # yarn: dims by the pair that makes beta turns, a ramp between them
    def pair(beta):
        return rotary * math.log(c["original"] / (beta * 2.0 * math.pi)) / (2.0 * math.log(THETA))
    lo, hi = max(math.floor(pair(c["beta_fast"])), 0), min(math.ceil(pair(c["beta_slow"])), rotary - 1)
    slow = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f * (1.0 - slow) + f / c["factor"] * slow, 0.1 * math.log(c["factor"]) + 1.0


def _rotated(x, cos, sin, rotary, interleaved):
    t = x.to(F32)
    a, b = (t[..., 0:rotary:2], t[..., 1:rotary:2]) if interleaved else t[..., :rotary].chunk(2, -1)
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, t[..., rotary:]], -1).to(x.dtype)


def _rotate(s):
    c = s["case"]
    if own:
        q, k = s["own"].rotate(s["q"], s["k"], s["pos"])
        return {"q": q, "k": k}
    f, factor = _frequencies(c["rotary"], c["scaling"])
    angle = s["pos"].to(F64)[..., None] * f
    cos, sin = ((factor * t).to(F32)[:, :, None] for t in (torch.cos(angle), torch.sin(angle)))
    return {n: _rotated(s[n], cos, sin, c["rotary"], c["interleaved"]) for n in ("q", "k")}


def _probabilities(x, temp):
    """softmax(x / temp) in 64 bits; where temp is 0, all of it on the first of the largest."""
    x = x.to(F64)
    V = x.shape[-1]
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / torch.where(temp > 0, temp, 1.0).to(F64)[:, None, None])
    first = torch.where(x == top, torch.arange(V, device=x.device), V).amin(-1, keepdim=True)
    hard = (torch.arange(V, device=x.device) == first).to(F64)
    return torch.where(temp[:, None, None] > 0, e / e.sum(-1, keepdim=True), hard)


def _verify(s):
    if own:
        from kv_cached_qwen3_gb300.draft import draft_verify
        got = draft_verify(s["target"], s["tokens"], s["u"], draft_logits=s["draft"], counts=s["count"],
                           temperatures=s["temp"])
        return dict(zip(("tokens", "accepted", "logprobs"), got))
    S, K1, V = s["target"].shape
    K = K1 - 1
    # in 64 bits: a uniform number next to a border of the distribution's sums decides for one token or the next
    p = _probabilities(s["target"], s["temp"])
    at = s["tokens"].long()[..., None]
    px = p[:, :K].gather(-1, at)[..., 0]
    if s["draft"] is not None:
        q = _probabilities(s["draft"], s["temp"])
        hard = torch.zeros_like(q).scatter_(-1, at, 1.0)       # a greedy draft is the token that it named
        q = torch.where(s["temp"][:, None, None] > 0, q, hard)
    else:
        q = torch.zeros_like(p[:, :K]).scatter_(-1, at, 1.0)
    qx = q.gather(-1, at)[..., 0]
    u = s["u"].to(F64)
    i = torch.arange(K, device="cuda")
    count = torch.full((S,), K, device="cuda") if s["count"] is None else s["count"].long()
    good = (u[:, :K] * qx < px) & (i < count[:, None])
    n = good.to(torch.int64).cumprod(-1).sum(-1)
    row = torch.arange(S, device="cuda")
    pn = p[row, n]
    left = (pn - q[row, n.clamp(max=K - 1)]).clamp(min=0.0)
    w = torch.where(((n < count) & (left.sum(-1) > 0))[:, None], left, pn)
    c = w.cumsum(-1)
    new = (c > u[:, K:] * c[:, -1:]).to(torch.int64).argmax(-1)
    j = torch.arange(K1, device="cuda")
    drafted = torch.nn.functional.pad(s["tokens"].long(), (0, 1))
    tokens = torch.where(j < n[:, None], drafted, torch.where(j == n[:, None], new[:, None], -1))
    lp = torch.log(p.gather(-1, tokens.clamp(min=0)[..., None])[..., 0])
    return {"tokens": tokens.to(torch.int32), "accepted": n.to(torch.int32),
            "logprobs": torch.where(tokens >= 0, lp, 0.0).to(F32)}


def run(state):
    return {"product": _product, "norm": _norm, "rotate": _rotate, "verify": _verify}[state["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["kind"] == "product":
        rows, n, k = case["rows"], case["n"], case["k"]
        weights = n * (2 if case["gated"] else 1)
        groups = -(-k // case["group"])
        size = weights * (k / 2 + groups * (2.5 if case["zeros"] else 2.0))
        size += rows * k * SIZE[case["x"]] + (rows * -(-k // 128) * 4 if case["x"] == "e4m3" else 0)
        return {"bytes": size + rows * n * SIZE[case["out"]] * (2 if case["residual"] else 1),
                "flops": 2.0 * rows * weights * k}
    if case["kind"] == "norm":
        one = SIZE[case["x"]] + SIZE[case["out"]] + (4 / (case["block"] or case["width"]) if case["out"] == "e4m3" else 0)
        one += 2 * SIZE[case["residual"]] if case["residual"] != "none" else 0
        return {"bytes": case["rows"] * case["width"] * one + 4 * case["width"], "flops": case["rows"] * case["width"] * 5}
    if case["kind"] == "rotate":
        rows = case["streams"] * case["rows"]
        dims = rows * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
        return {"bytes": dims * 2 * SIZE[case["x"]] + rows * 4, "flops": dims * 3}
    # rows of all drafts, as many as there are on average, and the one after them; of a greedy draft no probabilities
    S, K, V = case["seqs"], case["drafts"], case["vocab"]
    drafts = K / 2 if case["ragged"] else K
    soft = 0.5 if case["greedy"] else 1.0
    rows = S * (drafts + 1 + (drafts * soft if case["draft"] else 0))
    return {"bytes": rows * V * SIZE[case["x"]] + S * (K + 1) * 20, "flops": rows * V * 4}


# ------------------------------------------------------------------ the definition in 64 bits

def _product64(s, c):
    x = s["x"].to(F64)
    if s["xs"] is not None:
        block = torch.arange(c["k"], device="cuda") // 128
        x = x * s["xs"].to(F64)[:, block]
    ys = []
    for codes, scales, zeros in s["w"]:
        y = torch.zeros(c["rows"], c["n"], dtype=F64, device="cuda")
        for j in range(scales.shape[1]):                       # group by group
            lo, hi = j * c["group"], min((j + 1) * c["group"], c["k"])
            at = torch.arange(lo, hi, device="cuda")
            n = (codes[:, at // 2].long() >> (4 * (at % 2))) & 15
            n = n - (8 if zeros is None else zeros[:, j:j + 1].long())
            y += (x[:, lo:hi] @ n.to(F64).T) * scales[:, j].to(F64)
        ys.append(y)
    y = ys[0] if len(ys) == 1 else ys[0] * torch.sigmoid(ys[0]) * ys[1]
    return y if s["res"] is None else y + s["res"].to(F64)


def _norm64(s, c):
    t = s["x"].to(F64) + (0 if s["res"] is None else s["res"].to(F64))
    y = s["gain"].to(F64) * t * torch.rsqrt(t.pow(2).sum(-1, keepdim=True) / c["width"] + EPS)
    res = {"y": y, "sum": t if s["res"] is not None else None, "scales": None}
    if c["out"] == "e4m3":
        block = c["block"] or c["width"]
        tops = torch.stack([y[:, j:j + block].abs().amax(-1) for j in range(0, c["width"], block)], -1)
        res["scales"] = tops / 448
        v = y / (tops / 448)[:, torch.arange(c["width"], device="cuda") // block]
        # the nearest e4m3 value: a multiple of 2^(e - 3) with e at least -6, ties to even
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
        res["y"] = torch.round(v / step) * step
    return res


def _rotate64(s, c):
    R, C = c["rotary"], SCALINGS[c["scaling"]] or {"type": "none"}
    fs, factor = [], 1.0
    for j in range(R // 2):                                    # pair by pair
        base = THETA * C["factor"] ** (R / (R - 2)) if C["type"] == "ntk" else THETA
        f = math.exp(-2.0 * j / R * math.log(base))
        if C["type"] == "linear":
            f /= C["factor"]
        elif C["type"] == "smooth":                            # by the wavelength, in positions
            length, wave = C["original"], 2.0 * math.pi / f
            if wave > length / C["low"]:
                f /= C["factor"]
            elif wave > length / C["high"]:
                t = (length / wave - C["low"]) / (C["high"] - C["low"])
                f = (1.0 - t) * f / C["factor"] + t * f
        elif C["type"] == "yarn":
            ends = [R / 2 * math.log(C["original"] / b / 2 / math.pi, THETA) for b in (C["beta_fast"], C["beta_slow"])]
            lo, hi = max(0, math.floor(ends[0])), min(R - 1, math.ceil(ends[1]))
            t = min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3)))
            f, factor = f * ((1.0 - t) + t / C["factor"]), 1.0 + math.log(C["factor"]) / 10.0
        fs.append(f)
    f = torch.tensor(fs, dtype=F64, device="cuda")
    angle = s["pos"].to(F64)[..., None] * f
    turn = torch.polar(torch.full_like(angle, factor), angle)[:, :, None]
    res = {}
    for name in ("q", "k"):
        t = s[name].to(F64)
        y = t.clone()
        i = torch.arange(R // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
        z = torch.complex(t[..., a], t[..., b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
        res[name] = y
    return res


def _verify64(s, c):
    S, K1, V = s["target"].shape
    tokens = torch.full((S, K1), -1, dtype=torch.int64)
    accepted = torch.zeros(S, dtype=torch.int64)
    lps = torch.zeros(S, K1, dtype=F64)

    def soft(x, temp):
        if temp > 0:
            return torch.softmax(x.to(F64) / temp, -1)
        y = torch.zeros(V, dtype=F64, device="cuda")
        y[int((x == x.max()).nonzero()[0])] = 1.0
        return y
    for b in range(S):
        temp, u = float(s["temp"][b]), s["u"][b].double().cpu()
        count = K1 - 1 if s["count"] is None else int(s["count"][b])
        for i in range(count + 1):
            p = soft(s["target"][b, i], temp)
            w = p
            if i < count:
                x = int(s["tokens"][b, i])
                q = torch.zeros(V, dtype=F64, device="cuda")
                q[x] = 1.0
                if s["draft"] is not None and temp > 0:
                    q = soft(s["draft"][b, i], temp)
                if float(u[i]) * float(q[x]) < float(p[x]):
                    tokens[b, i], lps[b, i] = x, float(torch.log(p[x]))
                    accepted[b] += 1
                    continue
                w = torch.relu(p - q)
                if float(w.sum()) == 0:
                    w = p
            cum = torch.cumsum(w, 0)
            t = int(torch.searchsorted(cum, u[K1 - 1].cuda() * cum[-1], right=True))
            tokens[b, i], lps[b, i] = t, float(torch.log(p[t]))
            break
    return {"tokens": tokens.int(), "accepted": accepted.int(), "logprobs": lps}


def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _product64, "norm": _norm64, "rotate": _rotate64, "verify": _verify64}[case["kind"]](s, case)
