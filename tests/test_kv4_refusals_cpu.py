"""CPU: what the attention of f32 queries with bf16 results refuses before it touches a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from kv_cached_qwen3_gb300 import build, talker
    build.build()
    return talker.load_library()


def test_mixed_attention_refusals(lib):
    from kv_cached_qwen3_gb300.kv4 import _Cache

    def call(c, B=1, lens=64, max_len=10, n_q=4, q=256, out=512, scratch=None, n=0):
        return lib.talker_test_kv4_attend_mixed(c, B, lens, max_len, n_q, 1.0, q, out, scratch, n, None)
    good = _Cache(k=4096, v=8192, page_table=64, status=0, n_pages=8, n_streams=4, pages_per_stream=2, n_layers=3,
                  n_kv_heads=2, head_dim=64)
    at = ctypes.addressof(good)
    assert call(None) == 1
    for kw in (dict(B=5), dict(B=-1), dict(lens=None), dict(max_len=-1), dict(n_q=3), dict(n_q=18), dict(q=None), dict(q=258),
               dict(out=None), dict(out=513)):
        assert call(at, **kw) == 1, kw
    assert call(at, B=0) == 0
