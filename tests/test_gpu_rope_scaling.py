"""GPU: a Talker whose positions turn with scaled frequencies, against the oracle with the same."""
import numpy as np
import pytest

import layer_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SCALED = [dict(type="linear", factor=4.0), dict(type="ntk", factor=3.0), dict(type="smooth", factor=8.0, original=64, low=1.0, high=4.0),
          dict(type="yarn", factor=4.0, original=64, beta_fast=8.0, beta_slow=1.0)]


@pytest.mark.parametrize("scaling", SCALED, ids=lambda s: s["type"])
def test_prefill_and_decode(scaling, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300 import inputs
    from kv_cached_qwen3_gb300.talker import Talker, TalkerError
    from oracle import talker_oracle
    g = inputs.TINY
    w = inputs.make_weights(g, 3)

    def rope(x, positions, theta):
        return ref.rotate(torch.from_numpy(np.asarray(x)), torch.from_numpy(np.asarray(positions)), g.head_dim, theta, scaling, False)[0].numpy()
    plain = talker_oracle.Oracle(g, w)
    T0, n = 40, 3
    emb = inputs.make_embeddings(g, 3, 0, T0 + n)
    _, before = plain.forward_full(emb)
    monkeypatch.setattr(talker_oracle, "rope_neox", rope)
    _, want = talker_oracle.Oracle(g, w).forward_full(emb)
    tk = Talker(g, w)
    with pytest.raises(TalkerError):
        tk.set_rope_scaling(dict(scaling, factor=0.5))
    with pytest.raises(ValueError):
        tk.set_rope_scaling(dict(type="other"))
    tk.set_rope_scaling(scaling)
    tk.kv_init_batched(1, 64)
    with pytest.raises(TalkerError):
        tk.set_rope_scaling(scaling)                      # rows would be turned otherwise than those cached
    e = torch.from_numpy(emb).cuda()
    got = [tk.prefill(0, e[:T0])[1].cpu().numpy()]
    out = torch.empty(1, g.vocab, device="cuda")
    for t in range(n):
        tk.decode(e[T0 + t:T0 + t + 1].contiguous(), out)
        got.append(out[0].cpu().numpy())
    assert tk.sync_status() == 0
    tk.close()
    for a, b, c in zip(got, want[T0 - 1:], before[T0 - 1:]):
        assert np.linalg.norm(a - b) <= 1e-4 * np.linalg.norm(b)
        assert np.linalg.norm(a - c) > 1e-3 * np.linalg.norm(c)      # and it is not the plain rope
