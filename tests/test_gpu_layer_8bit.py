"""GPU: a decoder layer whose products take the norms' 8-bit rows, against 64 bits that take the same rows as they are."""
import math

import numpy as np
import pytest

import kv4_ref
import layer_ref as ref
import test_gpu_layer_run as run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def layer64(w, past, x, pos, rows):
    """One stream in 64 bits. rows: for each of the layer's three norms the values that its codes stand for. They have to be the
    norm's result (that of rows which f32 has moved by 1e-5 at most) within half a step of e4m3, and go on in its place."""
    def norm(t, g):
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + run.EPS) * g.double()
    at = iter(zip(rows, w.gains))

    def taken(t):
        (got, scales), gain = next(at)
        want = norm(t, gain)
        tops = want.view(-1, 32).abs().amax(-1)
        assert ((scales - tops / 448).abs() <= tops / 448 * 2e-5).all()
        spread = scales.repeat_interleave(32)
        # half a step of three bits and the leading one, or of the smallest steps, 2^-9; 1e-5 of s, its scale and the result
        assert ((got - want).abs() <= want.abs() * 2.0 ** -4 + spread * 2.0 ** -10 + 4e-5 * tops.repeat_interleave(32)).all()
        return got
    qkv = (taken(x) @ w.qkv64[0].T).view(run.HQ + 2 * run.HK, run.HD)
    q, k, v = norm(qkv[:run.HQ], w.gains[3]), norm(qkv[run.HQ:run.HQ + run.HK], w.gains[4]), qkv[run.HQ + run.HK:]
    p = torch.tensor([pos])
    q, k = (ref.rotate(t[None], p, run.HD, run.THETA, run.SCALING, False)[0][0] for t in (q, k))
    ks = np.stack([r[0] for r in past] + [k.numpy()])
    vs = np.stack([r[1] for r in past] + [v.numpy()])
    o = torch.from_numpy(kv4_ref.attend(q.numpy(), ks, vs, 1 / math.sqrt(run.HD)))
    past.append((kv4_ref.q4_roundtrip(k.numpy()), kv4_ref.q4_roundtrip(v.numpy())))
    x = x + o.reshape(-1) @ w.o64[0].T
    h = taken(x)
    g, u = h @ w.mlp64[0].T, h @ w.mlp64[1].T
    x = x + (g * torch.sigmoid(g) * u) @ w.down64[0].T
    return x, taken(x) @ w.head64[0].T


def test_a_layer_of_8_bit_rows(monkeypatch):
    """Steps of three streams. What is left between the two are f32 roundings, some hundred, 1e-5 of a row; and codes of cached rows that
    such a rounding moves by a step (a border within 1e-6 of a value: one in some 10^4 codes), 1/16 of one value in a row of the
    past: the bounds of the layer in f32."""
    from kv_cached_qwen3_gb300.kv4 import KV4Cache
    made = []
    norm8 = run.norm8

    def recorded(w, x, gain, residual=None):
        y, scales, s = norm8(w, x, gain, residual)
        made.append((y.float().double().cpu() * ref.by_block(scales.double().cpu(), 32, x.shape[1]), scales.double().cpu()))
        return y, scales, s
    monkeypatch.setattr(run, "norm8", recorded)
    w = run.Weights(1, True)
    B, T = 3, 9
    cache = KV4Cache(B, 128, 1, run.HK, run.HD)
    start = [0, 5, 40]
    past = [[] for _ in range(B)]
    for s in range(B):
        if start[s]:
            kv = [ref.rnd(100 + 2 * s + i, 1, 1, start[s], run.HK, run.HD) for i in range(2)]
            cache.write(*[t.cuda() for t in kv], stream0=s)
            for i in range(start[s]):
                past[s].append(tuple(kv4_ref.q4_roundtrip(t[0, 0, i].double().numpy()) for t in kv))
    for t in range(T):
        x = ref.rnd(200 + t, B, run.HID)
        pos = torch.tensor([a + t for a in start], dtype=torch.int32).cuda()
        made.clear()
        hid, lg = run.layer(w, cache, x.cuda(), pos, pos)
        assert len(made) == 3
        for s in range(B):
            want_h, want_l = layer64(w, past[s], x[s].double(), start[s] + t, [(y[s], d[s]) for y, d in made])
            for got, want in ((hid[s], want_h), (lg[s], want_l)):
                rel = float((got.double().cpu() - want).norm() / want.norm())
                assert rel < (2e-3 if t else 1e-5), (t, s, rel)
    assert cache.sync_status() == 0
