"""Workloads of the 4-bit KV cache operators and of beam selection.

A paged cache holds K and V rows as Q4_0 blocks: 32 dims share one fp16 scale d = -m / 8 (m the value of
largest magnitude, the first on ties) and hold 4-bit codes n = clamp(floor(8.5 - 8 x / m), 0, 15) that stand
for (n - 8) d. A page is 64 positions of every (layer, KV head): 64 * head_dim / 2 code bytes, then 64 *
(head_dim / 32) scales. Four kinds of case:

  write   rows written to the cache (quantized) and the same rows read back dense
  attend  one query row per stream attends its cached rows (decode), optionally with the step's own row
  select  beam search's choice of the best `width` of width * vocab continuations per sequence
  step    selection, the cache's streams reordered by the chosen parents, and every stream's rows handed out

`run` computes the plain form, or with `own` the framework's calls.
"""
import math

import torch

own = False

PAGE = 64
F32, F64 = torch.float32, torch.float64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    def write(name, layers, streams, rows, kv_heads, head_dim, dtype, past, ragged):
        return dict(name=name, kind="write", layers=layers, streams=streams, rows=rows, kv_heads=kv_heads,
                    head_dim=head_dim, dtype=dtype, past=past, ragged=ragged)

    def attend(name, streams, kv_heads, group, head_dim, length, dtype, fresh, ragged):
        return dict(name=name, kind="attend", streams=streams, kv_heads=kv_heads, group=group, head_dim=head_dim,
                    length=length, dtype=dtype, fresh=fresh, ragged=ragged)

    def select(name, seqs, width, vocab, dtype, ended):
        return dict(name=name, kind="select", seqs=seqs, width=width, vocab=vocab, dtype=dtype, ended=ended)

    def step(name, seqs, width, vocab, layers, kv_heads, head_dim, length, dtype):
        return dict(name=name, kind="step", seqs=seqs, width=width, vocab=vocab, layers=layers, kv_heads=kv_heads,
                    head_dim=head_dim, length=length, dtype=dtype)

    return [
        # one decode row of a single stream, all layers of the Talker stack
        write("write-row", 28, 1, 1, 8, 128, "f32", 130, False),
        # a padded batch of prompt chunks appended to one layer, from a bf16 projection
        write("write-chunks", 1, 4, 1999, 8, 64, "bf16", 777, True),
        # a whole prompt's state imported into every layer
        write("import-4096", 28, 1, 4096, 8, 128, "f32", 0, False),
        # the first steps after a short prompt: latency
        attend("attend-130", 1, 8, 2, 128, 130, "f32", True, False),
        # sixteen streams of very different lengths
        attend("attend-16-ragged", 16, 8, 2, 128, 2048, "f32", True, True),
        # one long stream
        attend("attend-32k", 1, 8, 2, 128, 32768, "f32", False, False),
        # wide groups of query heads, narrow heads, odd lengths
        attend("attend-g7-hd64", 7, 5, 7, 64, 5001, "bf16", False, True),
        # a full serving batch
        attend("attend-64x8k", 64, 8, 8, 128, 8192, "bf16", False, False),
        # one sequence over a codec vocabulary
        select("select-codec", 1, 4, 2048, "f32", False),
        # a batch over a text vocabulary, some beams already ended
        select("select-batch", 24, 8, 100003, "f32", True),
        # one short sequence's beams over a few layers
        step("step-4", 1, 4, 2048, 5, 8, 128, 100, "f32"),
        # several sequences of different lengths
        step("step-32", 4, 8, 4099, 5, 8, 128, 700, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["write", "attend", "attend", "select", "step"])
    hd = rng.choice([64, 128])
    dtype = rng.choice(["f32", "bf16"])
    if kind == "write":
        layers, streams, kvh = rng.randint(1, 28), rng.randint(1, 16), rng.randint(1, 16)
        most = max(1, min(4096, 28 * 4096 * 8 * 128 // (layers * streams * kvh * hd)))
        return dict(kind=kind, layers=layers, streams=streams, rows=_log(rng, 1, most), kv_heads=kvh, head_dim=hd,
                    dtype=dtype, past=rng.randint(0, 300), ragged=rng.random() < 0.5)
    if kind == "attend":
        streams, kvh, group = _log(rng, 1, 64), rng.randint(1, 16), rng.randint(1, 8)
        most = max(1, min(32768, 64 * 8 * 8192 * 128 // (streams * kvh * hd)))
        return dict(kind=kind, streams=streams, kv_heads=kvh, group=group, head_dim=hd, length=_log(rng, 1, most),
                    dtype=dtype, fresh=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if kind == "select":
        seqs, width = _log(rng, 1, 32), rng.randint(1, 16)
        most = max(256, min(150000, 24 * 8 * 100003 // (seqs * width)))
        return dict(kind=kind, seqs=seqs, width=width, vocab=_log(rng, 256, most), dtype=dtype,
                    ended=rng.random() < 0.5)
    seqs, width, layers, kvh = rng.randint(1, 6), rng.randint(1, 10), rng.randint(1, 8), rng.randint(1, 8)
    most = max(1, min(2000, 32 * 5 * 8 * 128 * 700 // (seqs * width * layers * kvh * hd)))
    return dict(kind=kind, seqs=seqs, width=width, vocab=_log(rng, 256, 5000), layers=layers, kv_heads=kvh,
                head_dim=hd, length=_log(rng, 1, most), dtype=dtype)


# ------------------------------------------------------------------ the cache's storage, plainly

def _quantize(x):
    """x [..., hd] -> codes uint8 [..., hd], scales fp16 [..., hd / 32]. In 64 bits: floor(8.5 - 8 x / m) decides
    between neighbouring codes, and 64 bits hold every such border of 32-bit inputs exactly."""
    b = x.to(F64).unflatten(-1, (-1, 32))
    a = b.abs()
    top = a.amax(-1, keepdim=True)
    at = torch.arange(32, device=x.device).expand_as(a)
    first = torch.where(a == top, at, 31).amin(-1, keepdim=True)
    m = b.gather(-1, first).clamp(-524032.0, 524032.0)
    n = torch.where(m == 0, 8.0, torch.floor(8.5 - 8.0 * b / m)).clamp(0, 15)
    return n.to(torch.uint8).flatten(-2), (m[..., 0] * -0.125).to(F32).to(torch.float16)


def _pack_k(n):
    """codes [..., 64, hd] -> bytes [..., 64 * hd / 2]: in a row, byte (c, b, j) holds dims 32 b + 8 c + 2 j, + 1."""
    n = n.unflatten(-1, (-1, 4, 4, 2))                        # b, c, j, nibble
    return (n[..., 0] | (n[..., 1] << 4)).transpose(-3, -2).flatten(-4)


def _pack_v(n):
    """codes [..., 64, hd] -> bytes: in a row, byte (g, b, e) holds dims 32 b + 4 g + 2 e, + 1."""
    n = n.unflatten(-1, (-1, 8, 2, 2))                        # b, g, e, nibble
    return (n[..., 0] | (n[..., 1] << 4)).transpose(-3, -2).flatten(-4)


def _tiles(n, d, pack):
    """codes [..., 64, hd], scales [..., 64, hd / 32] -> one tile's bytes [..., hd * 36]."""
    return torch.cat([pack(n), d.contiguous().view(torch.uint8).flatten(-2)], -1)


def _unpack(tiles, hd, is_v):
    """tile bytes [..., hd * 36] -> values f32 [..., 64, hd]."""
    nb = hd // 32
    codes, scales = tiles[..., :32 * hd], tiles[..., 32 * hd:].contiguous()
    b = codes.unflatten(-1, (PAGE, 8, nb, 2) if is_v else (PAGE, 4, nb, 4))
    n = torch.stack([b & 15, b >> 4], -1).transpose(-4, -3).flatten(-4, -2).flatten(-2)
    n = n.to(F32) - 8.0
    d = scales.view(torch.float16).to(F32).unflatten(-1, (PAGE, nb))
    return (n.unflatten(-1, (nb, 32)) * d[..., None]).flatten(-2)


def _dense(s, is_v, layers=slice(None)):
    """Every stream's rows of the pool, through the page table: [streams, layers, kv_heads, capacity, hd] f32."""
    pool, table, hd = s["vp" if is_v else "kp"], s["table"], s["head_dim"]
    x = _unpack(pool[:, layers][table.long()], hd, is_v)      # [streams, pages, layers, kv_heads, 64, hd]
    return x.permute(0, 2, 3, 1, 4, 5).flatten(3, 4)


# ------------------------------------------------------------------ prepare

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _lengths(seed, n, most, ragged):
    """Lengths of n streams: all `most`, or spread over 1/16 .. 1 of it with the longest first and a single row last."""
    if not ragged:
        return torch.full((n,), most, dtype=torch.int32, device="cuda")
    g = torch.Generator()
    g.manual_seed(int(seed) * 7919 + 17)
    x = (most * (1 / 16 + 15 / 16 * torch.rand(n, generator=g))).int().clamp(1, most)
    x[0] = most
    if n > 2:
        x[-1] = 1
    return x.cuda()


def _cache(s, seed, streams, capacity, layers, kv_heads, head_dim, filled, beams=False):
    """Pools of whole pages and a page table. Pages lie in any order; for beams, column j of the table holds pages
    r * pages_per_stream + j in any order of r."""
    pps = (capacity + PAGE - 1) // PAGE
    pages, tile = streams * pps, head_dim * 36
    g = _gen(seed, 1)
    if beams:
        r = torch.argsort(torch.rand(streams, pps, generator=g, device="cuda"), dim=0)
        table = r * pps + torch.arange(pps, device="cuda")
    else:
        table = torch.randperm(pages, generator=g, device="cuda").view(streams, pps)
    s.update(streams=streams, pps=pps, layers=layers, kv_heads=kv_heads, head_dim=head_dim,
             table=table.to(torch.int32).contiguous())
    for name, pack in (("kp", _pack_k), ("vp", _pack_v)):
        pool = torch.zeros(pages, layers, kv_heads, tile, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (layers * kv_heads * PAGE * head_dim))
        for p in range(0, pages if filled else 0, step):
            q = min(pages, p + step)
            pool[p:q] = _tiles(*_quantize(_normal(g, q - p, layers, kv_heads, PAGE, head_dim)), pack)
        s[name] = pool
    if own:
        from kv_cached_qwen3_gb300.kv4 import KV4Cache
        s["cache"] = KV4Cache.over(s["kp"], s["vp"], s["table"], head_dim)


def _beams(s, case, seed):
    g = _gen(seed, 2)
    S, W, V = case["seqs"], case["width"], case["vocab"]
    # what an output head gives: a few tokens of each row stand out
    x = 2.0 * _normal(g, S, W, V)
    s["logits"] = x.to(DTYPES[case.get("dtype", "f32")] if case["kind"] == "select" else F32)
    s["scores"] = -20.0 - 2.0 * torch.rand(S, W, generator=g, device="cuda", dtype=F32)
    s["eos"] = V // 3
    s["ended"] = None
    if case.get("ended"):
        s["ended"] = (torch.rand(S, W, generator=g, device="cuda") < 0.25).to(torch.int32)


def prepare(case, seed):
    s = {"kind": case["kind"], "dtype": DTYPES[case.get("dtype", "f32")]}
    g = _gen(seed, 3)
    if case["kind"] == "write":
        B, T, L, H, D = case["streams"], case["rows"], case["layers"], case["kv_heads"], case["head_dim"]
        _cache(s, seed, B, case["past"] + T, L, H, D, filled=False)
        s["k"] = _normal(g, L, B, T, H, D).to(s["dtype"])
        s["v"] = _normal(g, L, B, T, H, D).to(s["dtype"])
        s["start"] = torch.randint(0, case["past"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["count"] = _lengths(seed, B, T, True) if case["ragged"] else None
        s["ko"], s["vo"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    elif case["kind"] == "attend":
        B, H, G, D, n = case["streams"], case["kv_heads"], case["group"], case["head_dim"], case["length"]
        _cache(s, seed, B, n, 1, H, D, filled=True)
        s["q"] = _normal(g, B, H * G, D).to(s["dtype"])
        s["lens"] = _lengths(seed, B, n, case["ragged"])
        s["kn"] = _normal(g, B, H, D).to(s["dtype"]) if case["fresh"] else None
        s["vn"] = _normal(g, B, H, D).to(s["dtype"]) if case["fresh"] else None
        s["max_len"] = n
    else:
        _beams(s, case, seed)
        if case["kind"] == "step":
            S, W, n = case["seqs"], case["width"], case["length"]
            _cache(s, seed, S * W, n, case["layers"], case["kv_heads"], case["head_dim"], filled=True, beams=True)
            s["lens"] = _lengths(seed, S, n, S > 1).repeat_interleave(W)
            shape = (case["layers"], S * W, n, case["kv_heads"], case["head_dim"])
            s["ko"] = torch.zeros(shape, dtype=s["dtype"], device="cuda")
            s["vo"] = torch.zeros_like(s["ko"])
    return s


# ------------------------------------------------------------------ one pass

def _write(s):
    if own:
        s["cache"].write(s["k"], s["v"], start=s["start"], count=s["count"])
        s["cache"].read(s["ko"], s["vo"], start=s["start"], count=s["count"])
        return {"k": s["ko"], "v": s["vo"]}
    L, B, T, H, D = s["k"].shape
    i = torch.arange(T, device="cuda")
    valid = i < (s["count"][:, None] if s["count"] is not None else T)                  # [B or 1, T]
    b, i = (valid.expand(B, T)).nonzero(as_tuple=True)
    pos = s["start"].long()[b] + i
    page, row = s["table"].long()[b, pos // PAGE], pos % PAGE
    out = {}
    for name, pool, pack, is_v in (("k", s["kp"], _pack_k, False), ("v", s["vp"], _pack_v, True)):
        n, d = _quantize(s[name][:, b, i])                                              # [L, rows, H, D]
        codes = pool[..., :32 * D].unflatten(-1, (PAGE, D // 2))
        scales = pool[..., 32 * D:].unflatten(-1, (PAGE, D // 16))
        codes[page, :, :, row] = pack(n[..., None, :]).transpose(0, 1)
        scales[page, :, :, row] = d.view(torch.uint8).transpose(0, 1)
        # ... and the same rows back
        got = _unpack_rows(codes[page, :, :, row], scales[page, :, :, row], D, is_v)    # [rows, L, H, D]
        x = torch.zeros_like(s[name])
        x[:, b, i] = got.transpose(0, 1).to(x.dtype)
        out[name] = x
    return out


def _unpack_rows(codes, scales, hd, is_v):
    nb = hd // 32
    b = codes.unflatten(-1, (8, nb, 2) if is_v else (4, nb, 4))
    n = torch.stack([b & 15, b >> 4], -1).transpose(-4, -3).flatten(-4).to(F32) - 8.0
    d = scales.contiguous().view(torch.float16).to(F32)
    return (n.unflatten(-1, (nb, 32)) * d[..., None]).flatten(-2)


def _attend(s):
    if own:
        return s["cache"].attend(0, s["q"], s["lens"], k_new=s["kn"], v_new=s["vn"], max_len=s["max_len"])
    B, HQ, D = s["q"].shape
    H = s["kv_heads"]
    k, v = _dense(s, False, slice(0, 1))[:, 0], _dense(s, True, slice(0, 1))[:, 0]      # [B, H, capacity, D]
    q = s["q"].to(F32).view(B, H, HQ // H, D) * (1.0 / math.sqrt(D))
    w = q @ k.transpose(-1, -2)                                                         # [B, H, G, capacity]
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None]
    w = torch.where(seen[:, None, None], w, -math.inf)
    if s["kn"] is not None:
        w = torch.cat([w, (q * s["kn"].to(F32)[:, :, None]).sum(-1, keepdim=True)], -1)
        v = torch.cat([v, s["vn"].to(F32)[:, :, None]], 2)
    e = torch.exp(w - w.amax(-1, keepdim=True))
    return ((e @ v) / e.sum(-1, keepdim=True)).view(B, HQ, D).to(s["dtype"])


def _choose(s):
    """Tokens, parents (stream numbers), scores and ended flags of the best `width` continuations. In 64 bits: scores
    next to one another decide what is chosen."""
    S, W, V = s["logits"].shape
    x = s["logits"].to(F64)
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    c = x - lse + s["scores"].to(F64)[..., None]
    if s["ended"] is not None:
        stay = torch.where(torch.arange(V, device="cuda") == s["eos"], s["scores"].to(F64)[..., None], -math.inf)
        c = torch.where(s["ended"][..., None] != 0, stay, c)
    best, at = torch.sort(c.flatten(1), dim=-1, descending=True, stable=True)           # ties: the lowest index
    best, at = best[:, :W], at[:, :W]
    parent, token = at // V, at % V
    done = token == s["eos"]
    if s["ended"] is not None:
        done = done | (s["ended"].gather(1, parent) != 0)
    rows = torch.arange(S, device="cuda")[:, None] * W
    return token.to(torch.int32), (rows + parent).to(torch.int32), best.to(F32), done.to(torch.int32)


def _select(s):
    if own:
        from kv_cached_qwen3_gb300.beam import beam_select
        token, parent, best, done = beam_select(s["logits"], s["scores"], ended=s["ended"], eos_id=s["eos"])
    else:
        token, parent, best, done = _choose(s)
    return {"tokens": token, "parents": parent, "scores": best, "ended": done}


def _step(s):
    out = _select(s)
    parents = out["parents"].flatten()
    if own:
        after, lens = s["cache"].reorder(parents, s["lens"])
        after.read(s["ko"], s["vo"], count=lens)
        return {**out, "lens": lens, "k": s["ko"], "v": s["vo"]}
    p = parents.long()
    lens = s["lens"][p]
    n = s["ko"].shape[2]
    seen = (torch.arange(n, device="cuda") < lens[:, None])[None, :, :, None, None]
    for name, is_v in (("k", False), ("v", True)):
        x = _dense(s, is_v)[p][:, :, :, :n].permute(1, 0, 3, 2, 4)                      # [L, streams, n, H, D]
        out[name] = torch.where(seen, x, 0.0).to(s["dtype"])
    return {**out, "lens": lens}


def run(state):
    return {"write": _write, "attend": _attend, "select": _select, "step": _step}[state["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _lens_host(case):
    """The mean length of `_lengths`, which is what the sums below need (its draws differ by seed)."""
    n, most = case.get("streams", case.get("seqs", 1)), case.get("length", case.get("rows"))
    ragged = case.get("ragged", case["kind"] == "step" and case["seqs"] > 1)
    if not ragged:
        return n * most
    rest = n - 1 - (n > 2)
    return most + rest * max(1.0, most * 17 / 32) + (n > 2)


def work(case):
    size = {"f32": 4, "bf16": 2}[case.get("dtype", "f32")]
    if case["kind"] == "write":
        rows = _lens_host(case) * case["layers"] * case["kv_heads"] * case["head_dim"] * 2
        # the rows read and their codes and scales written; these read and the rows written
        return {"bytes": rows * 2 * (size + 0.5625), "flops": rows * 4}
    if case["kind"] == "attend":
        cached = _lens_host(case) * case["kv_heads"] * case["head_dim"]
        rows = case["streams"] * case["kv_heads"] * case["head_dim"] * size
        return {"bytes": cached * 2 * 0.5625 + rows * (2 * case["group"] + 2 * bool(case["fresh"])),
                "flops": cached * 4 * case["group"]}
    logits = case["seqs"] * case["width"] * case["vocab"]
    w = {"bytes": logits * (size if case["kind"] == "select" else 4) + case["seqs"] * case["width"] * 28,
         "flops": logits * 4}
    if case["kind"] == "step":
        rows = _lens_host(case) * case["width"] * case["layers"] * case["kv_heads"] * case["head_dim"] * 2
        w["bytes"] += rows * (size + 0.5625)
        w["flops"] += rows
    return w


# ------------------------------------------------------------------ the definition in 64 bits

def _value64(pool, page, row, layer, hd, is_v):
    """Stored rows (page, row: [n]) of a layer, for every KV head and dim, dim by dim from the layout: [n, H, hd]."""
    d = torch.arange(hd, device="cuda")
    b, r = d // 32, d % 32
    nb = hd // 32
    byte = (r // 4) * (2 * nb) + 2 * b + (r % 4) // 2 if is_v else (r // 8) * (4 * nb) + 4 * b + (r % 8) // 2
    t = pool[page, layer].long()                                                        # [n, H, tile]
    at = (row[:, None] * (hd // 2) + byte)[:, None].expand(-1, t.shape[1], -1)
    n = (t.gather(-1, at) >> (4 * (d % 2))) & 15
    lo = (32 * hd + (row[:, None] * nb + b) * 2)[:, None].expand(-1, t.shape[1], -1)
    bits = t.gather(-1, lo) + 256 * t.gather(-1, lo + 1)
    sign = 1.0 - 2.0 * (bits >> 15)
    e, f = (bits >> 10) & 31, (bits & 1023).to(F64)
    mag = torch.where(e == 0, f * 2.0 ** -24, (1.0 + f / 1024.0) * torch.exp2(e.to(F64) - 15.0))
    return (n - 8).to(F64) * sign * mag


def _half64(x):
    """The nearest fp16 value, in 64 bits: a multiple of 2^(e - 10), ties to even, with e at least -14."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-14)
    step = torch.exp2(e - 10)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "write":
        res = {}
        for name in ("k", "v"):
            x = s[name]
            y = torch.zeros(x.shape, dtype=F64, device="cuda")
            for layer in range(x.shape[0]):
                t = x[layer].to(F64).unflatten(-1, (-1, 32))
                hi, lo = t.max(-1, keepdim=True).values, t.min(-1, keepdim=True).values
                # on a tie of +m and -m the first of the two decides
                place = torch.arange(32, 0, -1, device="cuda")
                first_hi = ((t == hi) * place).amax(-1, keepdim=True)
                first_lo = ((t == lo) * place).amax(-1, keepdim=True)
                m = torch.where((hi > -lo) | ((hi == -lo) & (first_hi > first_lo)), hi, lo)
                codes = torch.minimum(torch.floor((17.0 * m - 16.0 * t) / (2.0 * m)), torch.tensor(15.0).cuda())
                y[layer] = ((codes - 8.0) * _half64(-m / 8.0)).flatten(-2)
            if s["count"] is not None:
                T = x.shape[2]
                y *= (torch.arange(T, device="cuda") < s["count"][:, None])[None, :, :, None, None]
            res[name] = y
        return res
    if kind == "attend":
        B, HQ, D = s["q"].shape
        H = s["kv_heads"]
        out = torch.zeros(B, HQ, D, dtype=F64, device="cuda")
        for b in range(B):
            n = int(s["lens"][b])
            pos = torch.arange(n, device="cuda")
            page = s["table"][b].long()[pos // PAGE]
            k = _value64(s["kp"], page, pos % PAGE, 0, D, False)
            v = _value64(s["vp"], page, pos % PAGE, 0, D, True)
            if s["kn"] is not None:
                k, v = torch.cat([k, s["kn"][b:b + 1].to(F64)]), torch.cat([v, s["vn"][b:b + 1].to(F64)])
            q = s["q"][b].to(F64).view(H, HQ // H, D)
            a = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(D), -1)
            out[b] = torch.einsum("hgn,nhd->hgd", a, v).reshape(HQ, D)
        return out
    S, W, V = s["logits"].shape
    scores = torch.empty(S, W, dtype=F64, device="cuda")
    parents = torch.empty(S, W, dtype=torch.long, device="cuda")
    tokens, done = torch.empty_like(parents), torch.empty_like(parents)
    for i in range(S):
        c = torch.log_softmax(s["logits"][i].to(F64), -1) + s["scores"][i].to(F64)[:, None]
        old = torch.zeros(W, dtype=torch.bool, device="cuda") if s["ended"] is None else s["ended"][i] != 0
        c[old] = -math.inf
        c[old, s["eos"]] = s["scores"][i].to(F64)[old]
        c = c.flatten()
        for j in range(W):                                    # the best left, and of equal ones the first
            top = c.max()
            at = (c == top).nonzero()[0, 0]
            scores[i, j], parents[i, j], tokens[i, j] = top, i * W + at // V, at % V
            done[i, j] = old[at // V] | (at % V == s["eos"])
            c[at] = -math.inf
    res = {"tokens": tokens.int(), "parents": parents.int(), "scores": scores, "ended": done.int()}
    if kind == "step":
        n = s["ko"].shape[2]
        p = parents.flatten()
        lens = s["lens"][p]
        res.update(lens=lens, k=torch.zeros(s["ko"].shape, dtype=F64, device="cuda"))
        res["v"] = torch.zeros_like(res["k"])
        for name, pool, is_v in (("k", s["kp"], False), ("v", s["vp"], True)):
            for r in range(S * W):
                pos = torch.arange(int(lens[r]), device="cuda")
                page = s["table"][p[r]].long()[pos // PAGE]
                for layer in range(case["layers"]):
                    res[name][layer, r, :len(pos)] = _value64(pool, page, pos % PAGE, layer, case["head_dim"], is_v)
    return res
