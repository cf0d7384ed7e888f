"""GPU checks of beam selection where a row's sum of exponentials decides: logits far from 0, and equal rows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def select():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300.beam import beam_select
    return beam_select


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def best_of(x, s):
    """One sequence in 64 bits: logits [W, V], scores [W] -> tokens, beams, scores. A row's largest logit is taken off
    before anything else is added, so that nothing is lost beside it."""
    x = np.where(x > -1e30, x, -np.inf)
    W, V = x.shape
    c = np.full((W, V), -np.inf)
    for w in range(W):
        m = x[w].max()
        if np.isfinite(m) and s[w] > -1e30:
            d = x[w] - m
            c[w] = d - np.log(np.exp(d).sum()) + s[w]
    at = np.argsort(-c.reshape(-1), kind="stable")[:W]
    return at % V, at // V, c.reshape(-1)[at]


def check(select, x, scores):
    """The choice itself, and scores: a sum of V terms (its exponentials within 2 units, pairs summed over at most
    V / 32 + 32 roundings), differences of logits within a unit of at most 2^-24 of 2^7 where a term counts, and a
    rounding of the score."""
    tok, par, best, _ = (t.cpu().numpy() for t in select(x, scores))
    S, W, V = x.shape
    for i in range(S):
        t, p, s = best_of(x[i].double().cpu().numpy(), scores[i].double().cpu().numpy())
        np.testing.assert_array_equal(par[i], i * W + p)
        np.testing.assert_array_equal(tok[i], t)
        fin = np.isfinite(s)
        np.testing.assert_array_equal(best[i][~fin], s[~fin])
        assert (np.abs(best[i][fin] - s[fin]) <= (V / 32 + 40 + 128) * 2.0 ** -24 + 2.0 ** -24 * np.abs(s[fin])).all(), (best[i], s)


@pytest.mark.parametrize("V,dt", [(300, "f32"), (300, "bf16"), (2048, "f32"), (5003, "bf16"), (40003, "f32")])
@pytest.mark.parametrize("size", [1e10, -1e10, 3e9, 1e12, -1e12, 1e20, -1e20, -1e29, -9.99e29, 1e30, 3e38])
def test_logits_far_from_0(select, V, dt, size):
    """Rows of one large value, of large values that differ, and of ordinary ones, as beams of one sequence."""
    W = 4
    x = rnd(1, 3, W, V) * 2
    base = torch.tensor(size).to(DT[dt]).item()
    x[0, :3] = base                                         # equal rows: -log V each
    x[1, 0] = base
    x[1, 1, : V // 2] = base                                # next to ordinary logits
    x[1, 2, 7:9] = base
    if abs(size) < 1e30:
        x[2] = base * (1 + (rnd(2, W, V) > 1) / 4.0)        # a quarter further out
    scores = -rnd(3, 3, W).abs()
    scores[0, 3] -= 50                                      # (its best tokens are no match for the equal rows')
    check(select, x.to(DT[dt]).cuda(), scores.cuda())


def test_a_masked_row_scores_no_better_than_its_beam(select):
    """All tokens at -1e10, a value that many programs mask with: each has -log V."""
    V = 1000
    x = rnd(1, 1, 2, V)
    x[0, 0] = -1e10
    best = select(x.cuda(), torch.zeros(1, 2).cuda())[2]
    assert float(best.max()) < 0


@pytest.mark.parametrize("V,dt", [(32001, "f32"), (50257, "f32"), (2049, "f32"), (2047, "bf16"), (50257, "bf16"), (12345, "bf16"),
                                  (151669, "f32"), (7, "f32")])
@pytest.mark.parametrize("W", [4, 7])
def test_equal_rows_are_taken_in_order(select, V, dt, W):
    """The same logits and score in every beam, in rows that lie on every place of 16 bytes: the best token of each
    beam is chosen, beam after beam, with one score."""
    for seed in range(3):
        x = (rnd(seed, V) * 2).to(DT[dt])
        x[V // 2] += 4
        rows = x.expand(2, W, V).contiguous().cuda()
        tok, par, best, _ = select(rows, torch.full((2, W), -1.5).cuda())
        want = torch.arange(2 * W).view(2, W)
        assert torch.equal(par.cpu().long(), want)
        assert (tok.cpu() == int(x.float().argmax())).all()
        assert (best == best[0, 0]).all()
        # some of the beams: those that are equal stay in order, between others
        rows[:, ::2] = (rnd(100 + seed, V) * 2).to(DT[dt]).cuda()
        check(select, rows, torch.full((2, W), -1.5).cuda())


def test_equal_rows_at_any_place(select):
    """Rows with a stride, in a tensor that starts anywhere: the same bits."""
    V, W = 5001, 5
    for dt in DT.values():
        x = (rnd(7, V) * 2).to(dt).cuda()
        got = []
        for off in range(9):
            for stride in (V, V + 3, V + 7):
                buf = torch.zeros(W * stride + off, dtype=dt, device="cuda")
                rows = buf[off:].view(1, W, stride)[..., :V]
                rows.copy_(x.expand(1, W, V))
                got.append([t.cpu() for t in select(rows, torch.zeros(1, W).cuda())])
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, got[0]))
