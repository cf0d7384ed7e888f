"""GPU: the verification of drafted tokens against 64 bits."""
import math

import numpy as np
import pytest

import layer_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def verify():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300.draft import draft_verify
    return draft_verify


def inputs(seed, S, K, V, dt, near=0.7):
    t = ref.rnd(seed, S, K + 1, V) * 2.5
    d = t[:, :K] + near * ref.rnd(seed + 1, S, K, V)
    e = -torch.log(ref.uni(seed + 2, S, K, V).clamp(min=1e-30))
    tokens = (d - torch.log(e)).argmax(-1).to(torch.int32) if K else torch.zeros(S, 0, dtype=torch.int32)
    return t.to(DT[dt]), d.to(DT[dt]), tokens, ref.uni(seed + 3, S, K + 1)


def check(verify, t, tokens, u, d=None, counts=None, temps=None):
    """Tokens and counts equal; log-probabilities: a difference of logits and the logarithm of a sum of V exponentials in
    f32, each a few units of 2^-22 and their roundings over a part."""
    cuda = [None if x is None else x.cuda() for x in (t, tokens, u, d, counts, temps)]
    out, n, lp = (x.cpu().numpy() for x in verify(*cuda[:3], draft_logits=cuda[3], counts=cuda[4], temperatures=cuda[5]))
    S, K1, V = t.shape
    for s in range(S):
        temp = 1.0 if temps is None else float(temps[s])
        w = ref.verify(t[s].double().numpy(), tokens[s].numpy(), u[s].double().numpy(), None if d is None else d[s].double().numpy(),
                       None if counts is None else int(counts[s]), temp)
        assert list(out[s]) == w[0] and n[s] == w[1], (s, list(out[s]), w)
        size = 1 + np.abs(w[2]) * 4 + (0 if not temp > 1e-20 else 1 / temp)
        assert (np.abs(lp[s] - np.array(w[2])) <= size * 2.0 ** -20).all(), (lp[s], w[2])
    return out, n, lp


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("S,K,V", [(1, 0, 1), (1, 1, 1), (2, 1, 2), (3, 3, 17), (5, 4, 64), (2, 7, 255), (1, 3, 2048), (7, 5, 1003), (3, 2, 32001), (2, 8, 50257), (1, 64, 300), (40, 2, 500)])
def test_sizes(verify, dt, S, K, V):
    for seed in (1, 20):
        t, d, tokens, u = inputs(seed, S, K, V, dt)
        check(verify, t, tokens, u, d)
        check(verify, t, tokens, u)
        counts = torch.randint(0, K + 1, (S,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        temps = 0.5 + ref.uni(seed, S)
        temps[::3] = 0.0
        check(verify, t, tokens, u, d, counts, temps)
        check(verify, t, tokens, u, None, counts, temps)


def test_every_count_is_reached(verify):
    """Enough sequences that each number of drafts is taken, and both kinds of draws."""
    t, d, tokens, u = inputs(5, 200, 4, 300, "f32", near=0.4)
    n = check(verify, t, tokens, u, d)[1]
    assert set(n) == {0, 1, 2, 3, 4}


def test_counts_temperatures_and_uniforms_out_of_range(verify):
    t, d, tokens, u = inputs(3, 8, 3, 100, "f32")
    counts = torch.tensor([-5, 0, 1, 2, 3, 4, 1000, -2 ** 31], dtype=torch.int32)
    u[0] = math.nan
    u[1] = -3.0
    u[2] = 7.0
    u[3] = math.inf
    u[4, 3] = 1.0
    u[5, :3] = 0.0
    temps = torch.tensor([1.0, 1e-3, 50.0, 1.0, -1.0, math.nan, 1e-30, math.inf])
    check(verify, t, tokens, u, d, counts)
    check(verify, t, tokens, u, None, counts)
    temps[7] = 1.0
    check(verify, t, tokens, u, d, counts, temps)


def test_temperature_without_bound_is_uniform(verify):
    """All tokens are as likely: u decides by itself."""
    t, d, tokens, u = inputs(3, 4, 0, 1000, "f32")
    out, _, lp = verify(t.cuda(), tokens.cuda(), u.cuda(), temperatures=torch.full((4,), math.inf).cuda())
    want = torch.floor(u[:, 0].double() * 1000).int()
    assert torch.equal(out[:, 0].cpu(), want) and (lp.cpu() + math.log(1000)).abs().max() < 1e-5


def test_masked_logits(verify):
    """Tokens that are masked out (-inf, the lowest value, NaN, -1e30) are never drawn, drafted ones are refused; rows of nothing else give -1."""
    t, d, tokens, u = inputs(9, 12, 2, 200, "f32")
    low = torch.finfo(torch.float32).min
    for i, v in enumerate((-math.inf, low, math.nan, -1e30)):
        t[i, :, 50:] = v
        d[i, :, 30:90] = v
    tokens[0, 0], tokens[1, 1] = 60, 199
    t[4, 1] = -math.inf
    t[5, 0] = low
    t[6, 2] = math.nan
    t[7, 1, 7] = math.inf
    d[8, 0] = -math.inf
    d[9, 1, 3] = math.inf
    t[10, :, 1:] = -math.inf
    t[11, 0, :] = -1e30
    u[10] = 0.999
    check(verify, t, tokens, u, d)
    check(verify, t, tokens, u)
    temps = torch.zeros(12)
    for i in range(12):
        tokens[i, 0] = int(torch.from_numpy(ref.unmask(t[i, 0])).argmax())
    check(verify, t, tokens, u, d, None, temps)
    out, n, _ = verify(t.cuda(), tokens.cuda(), u.cuda(), draft_logits=d.cuda())
    assert out[5].tolist() == [-1, -1, -1] and int(n[5]) == 0


def test_tokens_outside_the_vocabulary(verify):
    t, d, tokens, u = inputs(9, 4, 2, 200, "f32")
    tokens[0, 0], tokens[1, 0], tokens[2, 1], tokens[3, 1] = 200, -1, 2 ** 31 - 1, -2 ** 31
    check(verify, t, tokens, u, d)
    check(verify, t, tokens, u)
    check(verify, t, tokens, u, d, None, torch.zeros(4))


def test_equal_models_take_everything(verify):
    """p = q: any u below 1 takes a draft, however the rows lie, and a u of 1 none."""
    V, K = 5003, 4
    t, _, tokens, u = inputs(11, 3, K, V, "f32")
    u[:, :K] = 1.0 - 2.0 ** -24
    wide = torch.zeros(3, K, V + 5)
    wide[:, :, 3:3 + V] = t[:, :K]
    out, n, _ = verify(t.cuda(), tokens.cuda(), u.cuda(), draft_logits=wide.cuda()[:, :, 3:3 + V])
    assert (n == K).all() and torch.equal(out[:, :K].cpu(), tokens)
    u[:, 2] = 1.0
    n = verify(t.cuda(), tokens.cuda(), u.cuda(), draft_logits=wide.cuda()[:, :, 3:3 + V])[1]
    assert (n == 2).all()


def test_greedy_ties_go_to_the_lowest_index(verify):
    t, _, tokens, u = inputs(11, 2, 2, 3001, "f32")
    for i, at in enumerate(((5, 2999), (40, 41), (0, 3000))):
        t[:, i, list(at)] = 30.0
    tokens[0], tokens[1] = torch.tensor([5, 41]), torch.tensor([5, 40])
    out, n, lp = verify(t.cuda(), tokens.cuda(), u.cuda(), temperatures=torch.zeros(2).cuda())
    assert out.tolist() == [[5, 40, -1], [5, 40, 0]] and n.tolist() == [1, 2] and (lp == 0).all()


@pytest.mark.parametrize("scale", [1e-3, 30.0, 1e4, 1e20])
def test_logits_of_any_size(verify, scale):
    for dt in DT:
        t, d, tokens, u = inputs(2, 6, 3, 700, "f32")
        check(verify, (t * scale).to(DT[dt]), tokens, u, (d * scale).to(DT[dt]))
        check(verify, (t + 1e4).to(DT[dt]), tokens, u, (d - 1e4).to(DT[dt]))


def test_draws_are_where_64_bits_put_them(verify):
    """Uniform numbers a little below and above the borders between tokens: 2^-27 of the whole on either side, far over
    what the exponentials' 2^-31 and the number's own rounding can move (2^-24 of the number: small numbers are used)."""
    V = 4001
    t = ref.rnd(3, 1, 1, V) * 2.5
    p = ref.probabilities(t[0, 0].double().numpy(), 1.0)
    c = np.cumsum(p)
    at = [i for i in range(1, V) if c[i] < 2.0 ** -4][-60:]
    u = torch.tensor([[c[i] - 2.0 ** -27] for i in at] + [[c[i] + 2.0 ** -27] for i in at], dtype=torch.float32)
    want = [int(np.nonzero(c > float(x))[0][0]) for x in u[:, 0]]
    tt = t.expand(len(u), 1, V).contiguous()
    got = verify(tt.cuda(), torch.zeros(len(u), 0, dtype=torch.int32).cuda(), u.cuda())[0][:, 0].tolist()
    assert got == want


def test_rows_anywhere(verify):
    """Strides and starts of rows change nothing, not even a bit."""
    S, K, V = 3, 3, 1501
    t, d, tokens, u = inputs(4, S, K, V, "f32")
    for dt in DT.values():
        base = None
        for off, pad in ((0, 0), (1, 0), (3, 7), (2, 14), (8, 8)):
            tb, db = torch.zeros(S * (K + 1) * (V + pad) + off, dtype=dt).cuda(), torch.zeros(K * S * (V + pad) + off, dtype=dt).cuda()
            tv = torch.as_strided(tb, (S, K + 1, V), ((K + 1) * (V + pad), V + pad, 1), off)
            dv = torch.as_strided(db, (S, K, V), (V + pad, S * (V + pad), 1), off)        # drafts first, then sequences
            tv.copy_(t.to(dt))
            dv.copy_(d.to(dt))
            got = [x.cpu() for x in verify(tv, tokens.cuda(), u.cuda(), draft_logits=dv)]
            base = got if base is None else base
            assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
            assert (got[2] - base[2]).abs().max() < 1e-5


def test_empty_and_refused(verify):
    t, d, tokens, u = (x.cuda() for x in inputs(4, 2, 3, 50, "f32"))
    out, n, lp = verify(t[:0], tokens[:0], u[:0])
    assert out.shape == (0, 4) and n.shape == (0,) and lp.shape == (0, 4)
    one = torch.zeros(2, dtype=torch.int32).cuda()
    for args, kw in (((t.half(), tokens, u), {}), ((t[0], tokens, u), {}), ((t.cpu(), tokens, u), {}), ((t.transpose(1, 2), tokens, u), {}), ((t, tokens.long(), u), {}), ((t, tokens[:, :2], u), {}),
                     ((t, tokens, u[:, :3]), {}), ((t, tokens, u.double()), {}), ((t, tokens, u), dict(draft_logits=d[:, :2])), ((t, tokens, u), dict(draft_logits=d.bfloat16())),
                     ((t, tokens, u), dict(counts=one.long())), ((t, tokens, u), dict(counts=one[:1])), ((t, tokens, u), dict(temperatures=one)),
                     ((t, tokens, u), dict(temperatures=u)), ((torch.zeros(1, 66, 4).cuda(), torch.zeros(1, 65, dtype=torch.int32).cuda(), torch.zeros(1, 66).cuda()), {})):
        with pytest.raises(ValueError):
            verify(*args, **kw)
