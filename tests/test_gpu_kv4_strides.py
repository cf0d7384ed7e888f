"""GPU: rows whose K and V lie differently in memory where a dimension has one element."""
import numpy as np
import pytest

import kv4_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, 2, 3, 1, 64), (2, 1, 1, 2, 128), (1, 1, 130, 1, 128), (1, 3, 1, 1, 64)])
def test_strides_of_single_elements_do_not_count(shape):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300.kv4 import KV4Cache
    L, B, T, H, D = shape
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(shape, generator=g).cuda() for _ in (0, 1))
    odd = list(v.stride())
    for i, n in enumerate(shape):
        if n == 1:
            odd[i] += 4096 + 3
    w = torch.as_strided(v, shape, odd)
    assert w.stride() != k.stride()
    c = KV4Cache(B, T, L, H, D)
    out = [torch.empty_like(k), torch.as_strided(torch.empty_like(v), shape, odd)]
    for a, b in ((k, w), (w, k)):
        c.write(a, b)
        c.read(*out)
        for t, o in zip((a, b), out):
            np.testing.assert_array_equal(o.double().cpu().numpy(), ref.q4_roundtrip(t.double().cpu().numpy()))
    assert c.sync_status() == 0


def test_strides_that_differ_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300.kv4 import KV4Cache
    c = KV4Cache(2, 64, 1, 2, 64)
    k = torch.randn(1, 2, 3, 2, 64).cuda()
    for v in (k.transpose(2, 3).contiguous().transpose(2, 3), torch.randn(1, 2, 3, 2, 128).cuda()[..., :64]):
        with pytest.raises(ValueError):
            c.write(k, v)
