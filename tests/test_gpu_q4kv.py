"""GPU parity of the Q4_0 KV storage of a talker, and of reordering its streams.

A cached code may differ from the oracle's where a row's bf16-grade arithmetic moves a value across a border between
two codes, so each call is checked on rows that both sides share: the oracle takes the GPU's exported rows over
(they are what the codes stand for), and attends its own rows exactly, as the talker does.
"""
import numpy as np
import pytest

from kv_cached_qwen3_gb300 import inputs
from oracle import Oracle, OracleCache, decode_row_lazy_cache, q4_0_roundtrip
from parity_util import check_rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300 import talker
    talker.load_library()
    return torch.device("cuda", 0)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def host(t):
    return t.detach().float().cpu().numpy()


def geom(n_layers, **kw):
    return inputs.Geometry(**{**inputs.TALKER.__dict__, "n_layers": n_layers, "kv_dtype": "q4_0", **kw})


def export(tk, s, n, dtype=torch.float32):
    g = tk.g
    k = torch.empty(g.n_layers, g.n_kv_heads, n, g.head_dim, device="cuda", dtype=dtype)
    v = torch.empty_like(k)
    tk.kv_export(s, k, v, n)
    return k, v


def share(tk, oc, s):
    """The oracle's stream s holds the GPU's cached rows."""
    n = tk.cur_len(s)
    k, v = export(tk, s, n)
    oc.K[s][:, :, :n], oc.V[s][:, :, :n] = host(k), host(v)


def check_stored(tk, oc, s, lo, hi):
    """Exported rows lie within a code's step of the oracle's exact ones: half a step m / 8, a whole one at the far
    end, and 2% of m for the bf16 arithmetic that made the rows. oc stores its rows unquantized."""
    k, v = export(tk, s, hi)
    for got, want in ((host(k), oc.K[s][:, :, lo:hi]), (host(v), oc.V[s][:, :, lo:hi])):
        b = want.reshape(want.shape[:-1] + (-1, 32))
        m = np.abs(b).max(-1, keepdims=True)
        e = np.abs(got[:, :, lo:hi].astype(np.float64).reshape(b.shape) - b)
        assert (e <= m * (1 / 8 + 0.02)).all() and (e <= m * (1 / 16 + 0.02)).mean() > 0.98


@pytest.mark.parametrize("hd", [64, 128])
def test_import_codes_exact(cuda, hd):
    from kv_cached_qwen3_gb300.talker import Talker
    g = geom(2, head_dim=hd)
    w = inputs.make_weights(g, 72)
    tk = Talker(g, w)
    tk.kv_init_batched(2, 200)
    for L in (1, 7, 150):
        K = np.stack([inputs.make_kv_layer(g, 72, l, L)[0] for l in range(2)])
        V = np.stack([inputs.make_kv_layer(g, 72, l, L)[1] for l in range(2)])
        K[0, 0, 0] = 0.0
        tk.kv_import(1, dev(K), dev(V), L)
        k, v = export(tk, 1, L)
        np.testing.assert_array_equal(host(k), q4_0_roundtrip(K).astype(np.float32))
        np.testing.assert_array_equal(host(v), q4_0_roundtrip(V).astype(np.float32))
    assert tk.sync_status() == 0
    tk.close()


@pytest.mark.parametrize("hd,T0", [(128, 100), (128, 300), (128, 3), (64, 70)])
@pytest.mark.parametrize("mode", [pytest.param(2, id="gemv"), pytest.param(3, id="tensor-core")])
def test_prefill_then_decode(cuda, hd, T0, mode):
    from kv_cached_qwen3_gb300.talker import Talker
    g = geom(3, head_dim=hd)
    w = inputs.make_weights(g, 71)
    n = 4
    emb = inputs.make_embeddings(g, 71, 0, T0 + n)
    tk = Talker(g, w)
    tk.set_decode_mode(mode)
    tk.kv_init_batched(1, T0 + n + 1)
    o = Oracle(g, w)
    oc = OracleCache(o, 1, T0 + n + 1)
    hd_, lg, am = tk.prefill(0, dev(emb[:T0]))
    rh, rl = oc.prefill(0, emb[:T0])
    check_rows(host(hd_), rh[None], bf16=True, what="q4 prefill hidden")
    check_rows(host(lg), rl[None], bf16=True, what="q4 prefill logits")
    check_stored(tk, oc, 0, 0, T0)
    lgo, hdo = torch.empty(1, g.vocab, device="cuda"), torch.empty(1, g.hidden, device="cuda")
    for t in range(n):
        share(tk, oc, 0)
        e = emb[T0 + t:T0 + t + 1]
        tk.decode(dev(e), lgo, hdo)
        rh, rl = oc.decode(e)
        check_rows(host(hdo), rh, bf16=True, what="q4 decode %d hidden" % t)
        check_rows(host(lgo), rl, bf16=True, what="q4 decode %d logits" % t)
        check_stored(tk, oc, 0, T0 + t, T0 + t + 1)
    assert tk.sync_status() == 0
    tk.close()


@pytest.mark.parametrize("chunks", [[100, 70, 5, 16, 64], [300, 260]])
def test_appended_chunks(cuda, chunks):
    from kv_cached_qwen3_gb300.talker import Talker
    g = geom(2)
    w = inputs.make_weights(g, 53)
    emb = inputs.make_embeddings(g, 54, 0, sum(chunks))
    tk = Talker(g, w)
    tk.kv_init_batched(1, sum(chunks))
    oc = OracleCache(Oracle(g, w), 1, sum(chunks))
    at = 0
    for i, T in enumerate(chunks):
        part = emb[at:at + T]
        if i:
            share(tk, oc, 0)
        hd, lg, _ = tk.prefill(0, dev(part)) if i == 0 else tk.prefill_append(0, dev(part))
        rh, rl = oc.append_rows(0, part)
        check_rows(host(hd), rh[-1:], bf16=True, what="chunk %d hidden" % i)
        check_rows(host(lg), rl[-1:], bf16=True, what="chunk %d logits" % i)
        check_stored(tk, oc, 0, at, at + T)
        at += T
    assert tk.sync_status() == 0
    tk.close()


def test_batched_streams(cuda):
    from kv_cached_qwen3_gb300.talker import Talker
    g = geom(2)
    w = inputs.make_weights(g, 55)
    B, T = 5, 70
    emb = np.stack([inputs.make_embeddings(g, 55, 0, T + 2, stream=s) for s in range(B)])
    tk = Talker(g, w)
    tk.kv_init_batched(B, T + 2)
    oc = OracleCache(Oracle(g, w), B, T + 2)
    _, lg, _ = tk.prefill_batched(dev(emb[:, :T]))
    ref = np.stack([oc.prefill(s, emb[s, :T])[1] for s in range(B)])
    check_rows(host(lg), ref, bf16=True, what="q4 batched prefill")
    tk.rewind(1, 40)          # streams of different lengths
    oc.rewind(1, 40)
    for t in range(2):
        for s in range(B):
            share(tk, oc, s)
        e = emb[:, T + t] if t else emb[:, T]
        lg, _, _ = tk.decode(dev(e))
        _, rl = oc.decode(e)
        check_rows(host(lg), rl, bf16=True, what="q4 batched decode %d" % t)
    assert tk.sync_status() == 0
    tk.close()


@pytest.mark.parametrize("L", [3000, 8192])
def test_long_context_decode(cuda, L):
    from kv_cached_qwen3_gb300.talker import Talker
    g = geom(4)
    w = inputs.make_weights(g, 4)
    o = Oracle(g, w)
    K, V = (np.stack(x) for x in zip(*(inputs.make_kv_layer(g, 4, l, L) for l in range(4))))
    stored = [(q4_0_roundtrip(K[l]), q4_0_roundtrip(V[l])) for l in range(4)]
    emb = inputs.make_embeddings(g, 4, L, L + 1)
    rh, rl = decode_row_lazy_cache(o, emb[0], L, lambda l: stored[l])
    tk = Talker(g, w)
    tk.kv_init_batched(1, L + 1)
    tk.kv_import(0, dev(K), dev(V), L)
    lg, hd = torch.empty(1, g.vocab, device="cuda"), torch.empty(1, g.hidden, device="cuda")
    for mode in (2, 3):
        tk.set_decode_mode(mode)
        tk.rewind(0, L)
        tk.decode(dev(emb), lg, hd)
        check_rows(host(hd), rh[None], bf16=True, what="q4 L=%d mode %d hidden" % (L, mode))
        check_rows(host(lg), rl[None], bf16=True, what="q4 L=%d mode %d logits" % (L, mode))
    assert tk.sync_status() == 0
    tk.close()


def test_frame_runs_like_its_steps(cuda):
    """The whole-frame graph over Q4_0 storage gives what its prefill and steps give one by one."""
    from kv_cached_qwen3_gb300.talker import Talker
    g = geom(2, vocab=2048)
    w = inputs.make_weights(g, 9)
    tables = [torch.randn(g.vocab, g.hidden, device="cuda").bfloat16() for _ in range(3)]
    emb = dev(inputs.make_embeddings(g, 9, 0, 2))
    tk = Talker(g, w)
    tk.kv_init_batched(1, 16)
    tk.set_code_tables(tables, True)
    codes = torch.empty(4, dtype=torch.int32, device="cuda")
    logits = torch.empty(4, g.vocab, device="cuda")
    tk.frame(emb, [0, 1, 2], codes, logits)
    tk2 = Talker(g, w)
    tk2.kv_init_batched(1, 16)
    tk2.set_decode_mode(2)
    _, lg, _ = tk2.prefill(0, emb)
    check_rows(host(logits[0]), host(lg)[None], bf16=True, what="frame prefill")
    for i in range(3):
        lg, _, _ = tk2.decode(tables[i][codes[i:i + 1].long()].float().contiguous())
        check_rows(host(logits[i + 1]), host(lg), bf16=True, what="frame step %d" % i)
    assert tk.sync_status() == 0
    tk.close()
    tk2.close()


STORAGE = [("f32", dict(weight_dtype="f32", kv_dtype="f32", n_q_heads=4, n_kv_heads=2, head_dim=32, hidden=128,
                        intermediate=384, vocab=256)),
           ("bf16", dict(kv_dtype="bf16")), ("q8_0", dict(kv_dtype="q8_0")), ("q4_0", dict(kv_dtype="q4_0")),
           ("q4_0-hd64", dict(kv_dtype="q4_0", head_dim=64))]


@pytest.mark.parametrize("kw", [pytest.param(kw, id=name) for name, kw in STORAGE])
def test_reorder(cuda, kw):
    """Two groups of three streams reordered twice: every stream holds its parent's rows, attends them, and what is
    written to it afterwards (a step, a rewound stream, a prefill, an import) touches no other."""
    from kv_cached_qwen3_gb300.talker import Talker, TalkerError
    g = geom(2, **kw)
    w = inputs.make_weights(g, 31)
    edt = torch.bfloat16 if g.kv_dtype == "bf16" else torch.float32
    lens = [130, 130, 130, 64, 64, 64]
    tk, ref = Talker(g, w), Talker(g, w)
    for t in (tk, ref):
        t.kv_init_batched(7, 200)
    rows = []
    for s, n in enumerate(lens + [50]):
        k, v = (torch.randn(g.n_layers, g.n_kv_heads, n, g.head_dim, device="cuda").to(edt) for _ in (0, 1))
        tk.kv_import(s, k, v, n)
        rows.append(export(tk, s, n, edt))

    def same(s, want):
        n = tk.cur_len(s)
        got = export(tk, s, n, edt)
        assert n == want[0].shape[2] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), s
    for parents in ([2, 2, 0, 4, 3, 4], [0, 1, 1, 5, 5, 5]):
        tk.kv_reorder(torch.tensor(parents, dtype=torch.int32).cuda(), 2, 3)
        rows = [rows[p] for p in parents] + rows[6:]
        for s in range(7):
            same(s, rows[s])
    # a step on every stream, against a talker whose streams were imported
    for s in range(7):
        ref.kv_import(s, *rows[s], rows[s][0].shape[2])
    e = torch.randn(7, g.hidden, device="cuda")
    a, b = tk.decode(e)[0], ref.decode(e)[0]
    check_rows(host(a), host(b), bf16=g.weight_dtype == "bf16", what="step after reordering")
    rows = [export(ref, s, ref.cur_len(s), edt) for s in range(7)]
    if g.kv_dtype in ("f32", "bf16"):          # (a code may flip between the two, a plain row only rounds)
        for s in range(7):
            got = export(tk, s, tk.cur_len(s), edt)
            assert torch.allclose(got[0].float(), rows[s][0].float(), atol=3e-2, rtol=3e-2)
    rows = [export(tk, s, tk.cur_len(s), edt) for s in range(7)]
    # cut a stream inside a page that others share, and write to it
    tk.rewind(1, 10)
    rows[1] = tuple(x[:, :, :10].contiguous() for x in rows[1])
    for s in range(7):
        same(s, rows[s])
    n = 3
    tk.decode(torch.randn(n, g.hidden, device="cuda"))
    for s in range(7):
        if s < n:
            got = export(tk, s, rows[s][0].shape[2], edt)
            assert torch.equal(got[0], rows[s][0]) and torch.equal(got[1], rows[s][1]), s
        else:
            same(s, rows[s])
    rows = [export(tk, s, tk.cur_len(s), edt) for s in range(7)]
    # ... a prefill and an import over streams that share pages
    tk.prefill(4, torch.randn(70, g.hidden, device="cuda"))
    k, v = (torch.randn(g.n_layers, g.n_kv_heads, 100, g.head_dim, device="cuda").to(edt) for _ in (0, 1))
    tk.kv_import(5, k, v, 100)
    for s in (0, 1, 2, 3, 6):
        same(s, rows[s])
    with pytest.raises(TalkerError):          # lengths of a group differ
        tk.kv_reorder(torch.zeros(6, dtype=torch.int32).cuda(), 2, 3)
    if g.weight_dtype == "bf16":
        for s in range(1, 7):
            tk.rewind(s, 0)
        lg, rl = tk.prefill_batched(torch.randn(7, 70, g.hidden, device="cuda"))[1], None
        assert torch.isfinite(lg).all()
        assert all(tk.cur_len(s) == 70 for s in range(7))
        k = torch.stack([export(tk, s, 70, edt)[0] for s in range(7)])
        assert all(not torch.equal(k[i], k[j]) for i in range(7) for j in range(i))
    assert tk.sync_status() == 0
    # a parent outside its group is reported and counts as the stream itself
    if g.weight_dtype == "bf16":
        before = [export(tk, s, 70, edt) for s in range(6)]
        tk.kv_reorder(torch.tensor([0, 3, 99, 3, 4, -1], dtype=torch.int32).cuda(), 2, 3)
        for s in range(6):
            same(s, before[s])
        assert tk.sync_status() == 8
    tk.close()
    ref.close()


def test_beam_search_over_a_talker(cuda):
    """Beams as streams: decode, select, reorder. A beam's logits are those of its tokens replayed on their own."""
    from kv_cached_qwen3_gb300.beam import beam_select
    from kv_cached_qwen3_gb300.talker import Talker
    g = geom(2, vocab=2048)
    w = inputs.make_weights(g, 77)
    W, T0, steps = 4, 62, 6
    table = torch.randn(g.vocab, g.hidden, device="cuda")
    prompt = torch.randn(T0, g.hidden, device="cuda")
    tk = Talker(g, w)
    tk.kv_init_batched(W, T0 + steps + 1)
    for s in range(W):
        _, lg, _ = tk.prefill(s, prompt)
    logits = lg[None].expand(W, -1).contiguous()
    scores = torch.tensor([[0.0] + [float("-inf")] * (W - 1)]).cuda()
    history = torch.zeros(W, 0, dtype=torch.long, device="cuda")
    for t in range(steps):
        tok, par, scores, _ = beam_select(logits[None] * 8, scores)
        p = par.flatten().long()
        tk.kv_reorder(par.flatten(), 1, W)
        history = torch.cat([history[p], tok.flatten().long()[:, None]], 1)
        logits = tk.decode(table[tok.flatten().long()].contiguous())[0].clone()
    assert len({tuple(h.tolist()) for h in history}) == W
    alone = Talker(g, w)
    alone.kv_init_batched(W, T0 + steps + 1)
    for s in range(W):
        alone.prefill(s, prompt)
    for t in range(steps):
        want = alone.decode(table[history[:, t]].contiguous())[0]
    check_rows(host(logits), host(want), bf16=True, what="beams")
    assert tk.sync_status() == 0
    tk.close()
    alone.close()


def test_refusals(cuda):
    from kv_cached_qwen3_gb300.talker import Talker, TalkerError
    g = geom(1)
    for bad in ({"weight_dtype": "f32"}, {"head_dim": 32, "intermediate": 384}):
        gb = inputs.Geometry(**{**g.__dict__, **bad})
        with pytest.raises(TalkerError):
            Talker(gb, inputs.make_weights(gb, 73))
    g64 = geom(1, head_dim=64)
    tk = Talker(g64, inputs.make_weights(g64, 73))
    par = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TalkerError):
        tk.kv_reorder(par, 1, 2)              # no cache yet
    tk.kv_init_batched(2, 100)
    tk.prefill(0, torch.randn(20, g64.hidden, device="cuda"))
    with pytest.raises(TalkerError):          # appends over quantized rows need head_dim 128
        tk.prefill_append(0, torch.randn(20, g64.hidden, device="cuda"))
    with pytest.raises(TalkerError):
        tk.kv_reorder(par, 1, 2)              # lengths differ
    with pytest.raises(TalkerError):
        tk.kv_reorder(torch.zeros(3, dtype=torch.int32, device="cuda"), 1, 3)
    with pytest.raises(ValueError):
        tk.kv_reorder(par.long(), 1, 2)
    tk.close()
