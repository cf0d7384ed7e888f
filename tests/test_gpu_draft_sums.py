"""GPU: the verification of drafts over very long vocabularies, and over rows whose logits are the least that count."""
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


def row(kind, vocab, dt):
    i = torch.arange(vocab, device="cuda", dtype=torch.float32) / vocab
    if kind == "equal":
        x = torch.full((vocab,), -0.1, device="cuda")
        x[5] = 0.0
    elif kind == "rising":
        x = 3 * i - 2
    elif kind == "falling":
        x = -3 * i
    elif kind == "steep":
        x = 40 * i
    else:
        x = torch.randn(vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    return x.to(DT[dt])


def logs64(x):
    """log p of every token, in 64 bits."""
    x = x.double()
    return x - torch.logsumexp(x, 0)


# u q / p of a taken draft, and of a refused one: a decision is exact, or made by f32 sums with 1e-4 of room on both sides
NEAR = (1 - 2e-4, 1 + 2e-4, 1 - 2e-6, 1 + 2e-6)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "steep", "random"])
@pytest.mark.parametrize("n_seq,vocab", [(4, 1 << 26), (3300, 1 << 20), (4, 999983)])
def test_long_rows(verify, dt, kind, n_seq, vocab):
    """Rows of 2^26 logits, and of 2^20 with so many sequences that a warp goes over a row by itself; the same row for all.
    log p of a taken draft: a sum whose error does not grow with the row, of exponentials within 2^-22 whose arguments
    (58 at most, three roundings) add 58 * 3 * 2^-24 = 1e-5, and the result's own rounding."""
    x = row(kind, vocab, dt)
    token = vocab - 77
    lp = float(logs64(x)[token])
    target = x.expand(n_seq, 2, vocab)
    tokens = torch.full((n_seq, 1), token, dtype=torch.int32, device="cuda")
    near = torch.tensor(NEAR, dtype=torch.float64).repeat(n_seq // 4 + 1)[:n_seq]
    u = torch.full((n_seq, 2), 0.25, dtype=torch.float32)
    u[:, 0] = (math.exp(lp) * near).float()       # (rounded by 2^-24 at most)
    out, n, lps = verify(target, tokens, u.cuda())
    want = (near < 1).to(torch.int32)
    assert torch.equal(n.cpu(), want), (kind, (n.cpu() != want).nonzero().flatten().tolist()[:8])
    taken = want.bool()
    assert (out.cpu()[taken, 0] == token).all()
    assert ((lps.cpu()[taken, 0].double() - lp).abs() <= 1e-5 + abs(lp) * 2.0 ** -23).all(), (kind, lps.cpu()[taken, 0], lp)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_long_rows_of_both_models(verify, dt):
    vocab = 1 << 24
    p, q = row("equal", vocab, dt), row("rising", vocab, dt)
    token = vocab - 77
    ratio = math.exp(float(logs64(p)[token]) - float(logs64(q)[token]))
    assert ratio < 1
    u = torch.full((4, 2), 0.5, dtype=torch.float32)
    u[:, 0] = (ratio * torch.tensor(NEAR, dtype=torch.float64)).float()
    tokens = torch.full((4, 1), token, dtype=torch.int32, device="cuda")
    _, n, _ = verify(p.expand(4, 2, vocab), tokens, u.cuda(), draft_logits=q.expand(4, 1, vocab))
    assert n.tolist() == [1, 0, 1, 0]


LEAST = float(np.nextafter(np.float32(-1e30), np.float32(0)))    # the least logit that counts


@pytest.mark.parametrize("temp", [0.0, 1e-19, 1.0, 1e18, math.inf])
@pytest.mark.parametrize("vocab", [1, 3, 700, 50001])
def test_least_logits(verify, temp, vocab):
    """Rows whose only logits that count are the least that do: one, two, and beside masked values and NaNs."""
    S = 6
    t = torch.full((S, 2, vocab), -1e30)
    at = vocab // 2
    t[0, :, at] = LEAST
    t[1, :, 0] = t[1, :, at] = LEAST
    t[2] = LEAST
    t[3, :, at] = float(np.nextafter(np.float32(LEAST), np.float32(0)))
    t[4, :, 0], t[4, :, at] = math.nan, LEAST
    # (row 5: none)
    tokens = torch.full((S, 1), at, dtype=torch.int32)
    u = torch.tensor([[0.4, 0.6]]).repeat(S, 1)
    d = torch.full((S, 1, vocab), -math.inf)
    d[:, 0, at] = LEAST
    temps = torch.full((S,), temp)
    for draft in (None, d):
        out, n, lp = (x.cpu() for x in verify(t.cuda(), tokens.cuda(), u.cuda(), draft_logits=None if draft is None else draft.cuda(), temperatures=temps.cuda()))
        for s in range(S):
            # (temperatures above 1e18 count as it; so do they to the reference, whose rows hold equal logits or masked ones)
            want = ref.verify(t[s].double().numpy(), tokens[s].numpy(), u[s].double().numpy(), None if draft is None else draft[s].double().numpy(),
                              temp=min(temp, 1e18))
            assert out[s].tolist() == want[0] and int(n[s]) == want[1], (s, out[s], want)
            assert (lp[s].double() - torch.tensor(want[2])).abs().max() <= 2e-5


@pytest.mark.parametrize("top,rest", [(9.0, -0.9921875 * 2.0 ** -21), (12.0, -0.9921875 * 2.0 ** -21), (9.0, 0.4921875 * 2.0 ** -20), (5.0, -0.9921875 * 2.0 ** -22)])
def test_bf16_logits_far_apart_in_size(verify, top, rest):
    """Logits next to 0 under a larger one, whose differences have more bits than f32: a draw is that of the same logits in f32.
    (Half of them are 0 and lose nothing; without what the difference rounds off of the others, 2^-22 or 2^-21, draws
    among 2^24 are a token or more away.)"""
    S, vocab = 64, 1 << 24
    x = torch.zeros(vocab, dtype=torch.bfloat16, device="cuda")
    x[1:vocab // 2] = rest
    x[0] = top
    assert float(x[1]) == rest
    u = (0.2 + 0.6 * torch.arange(S, dtype=torch.float32) / S)[:, None].cuda()
    none = torch.zeros(S, 0, dtype=torch.int32, device="cuda")
    out, _, lp = verify(x.expand(S, 1, vocab), none, u)
    same, _, lp32 = verify(x.float().expand(S, 1, vocab), none, u)
    assert torch.equal(out, same)
    assert (lp - lp32).abs().max() <= 1e-6


def behind(u, first, parts):
    """Which token a draw meets, as a real number of tokens behind the first: `first` is the first token's weight, parts the
    (tokens, weight of each) that follow. Also how many of its tokens the whole sum is."""
    total = first + sum(n * w for n, w in parts)
    left, at = u * total - first, 0.0
    if left < 0:
        return -1.0, 1.0
    for n, w in parts:
        if left < n * w:
            return at + left / w, total / w
        left, at = left - n * w, at + n
    return at, total / parts[-1][1]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("top,vocab", [(16.0, 1 << 24), (16.0, 1 << 26), (12.0, 1 << 26), (20.0, 1 << 26), (10.0, 151936), (30.0, 262144)])
def test_a_large_logit_before_many_small_ones(verify, dt, top, vocab):
    """One token with most of a long row, which the others have the rest of: draws against 64 bits. An exponential is off by 2^-29 of itself,
    a sum by what its units cut off, 2^-28: 2^-27 of the sum, in tokens."""
    x = torch.full((vocab,), -0.5, dtype=DT[dt], device="cuda")
    x[vocab // 2:] = 0
    x[0] = top
    S = 64
    total = 1 + math.exp(-top) * (vocab // 2) + math.exp(-top - 0.5) * (vocab // 2 - 1)
    u = ((1 / total) + (1 - 1 / total) * (0.02 + 0.96 * torch.arange(S, dtype=torch.float64) / S)).float()[:, None]
    out, _, lp = verify(x.expand(S, 1, vocab), torch.zeros(S, 0, dtype=torch.int32, device="cuda"), u.cuda())
    for s in range(S):
        at, tokens = behind(float(u[s, 0]), 1.0, [(vocab // 2 - 1, math.exp(-top - 0.5)), (vocab // 2, math.exp(-top))])
        near, got = tokens * 2.0 ** -27, int(out[s, 0])
        assert math.floor(at - near) <= got - 1 <= math.floor(at + near), (s, got, at, near)
        if got > 0:
            assert abs(float(lp[s, 0]) - (float(x[got]) - top - math.log(total))) <= 1e-5


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("gone,small,vocab", [(0, 40.0, 100003), (77, 40.0, 1000), (100002, 25.0, 100003), (5, 47.0, 2048), (5, 47.0, 151936), (0, 30.0, 1 << 24)])
def test_what_is_left_of_a_refused_token(verify, dt, gone, small, vocab):
    """A certain draft that has nearly all of p, refused by u = 1: the next token is one of the others, in their proportions, not the draft."""
    x = torch.full((vocab,), -small, dtype=DT[dt], device="cuda")
    x[vocab // 2:] = -small + 1
    x[gone] = 0
    S = 32
    u = torch.ones(S, 2)
    u[:, 1] = 0.01 + 0.98 * torch.arange(S) / S
    tokens = torch.full((S, 1), gone, dtype=torch.int32)
    out, n, lp = (t.cpu() for t in verify(x.expand(S, 2, vocab), tokens.cuda(), u.cuda()))
    assert (n == 0).all() and (out[:, 1] == -1).all()
    half = vocab // 2
    parts = [(half - (gone < half), math.exp(-1.0)), (vocab - half - (gone >= half), 1.0)]
    for s in range(S):
        at, of = behind(float(u[s, 1]), 0.0, parts)
        near = of * 2.0 ** -27
        got = int(out[s, 0])
        assert got != gone
        assert math.floor(at - near) <= got - (got > gone) <= math.floor(at + near), (s, got, at, near)
        total = 1 + sum(n * w for n, w in parts) * math.exp(1 - small)
        assert abs(float(lp[s, 0]) - (float(x[got]) - math.log(total))) <= 1e-5


def test_a_draft_near_its_border_beside_a_large_logit(verify):
    """u q next to p, both rows with most on one token and 2^24 small ones: decided by sums of both rows as 64 bits decide."""
    vocab, top = 1 << 24, 17.0
    p = torch.zeros(vocab, device="cuda")
    p[0] = top
    q = torch.full((vocab,), 1.0, device="cuda")
    q[1] = top + 0.5
    token = 12345
    lp, lq = float(logs64(p)[token]), float(logs64(q)[token])
    ratio = math.exp(lp - lq)
    assert ratio < 1
    near = torch.tensor([1 - 2e-7, 1 + 2e-7, 1 - 1e-6, 1 + 1e-6], dtype=torch.float64)
    u = torch.full((4, 2), 0.5)
    u[:, 0] = (ratio * near).float()
    tokens = torch.full((4, 1), token, dtype=torch.int32, device="cuda")
    _, n, _ = verify(p.expand(4, 2, vocab), tokens, u.cuda(), draft_logits=q.expand(4, 1, vocab))
    assert n.tolist() == [int(float(u[i, 0]) < ratio) for i in range(4)] == [1, 0, 1, 0]
