"""CPU checks of the 4-bit cache's C-ABI: what it refuses before it touches a GPU, and the definitions it is held to."""
import ctypes

import numpy as np
import pytest

import kv4_ref as ref


@pytest.fixture(scope="module")
def lib():
    from kv_cached_qwen3_gb300 import build, talker
    build.build()
    return talker.load_library()


def cache(**kw):
    from kv_cached_qwen3_gb300.kv4 import _Cache
    f = dict(k=4096, v=8192, page_table=64, status=0, n_pages=8, n_streams=4, pages_per_stream=2, n_layers=3, n_kv_heads=2,
             head_dim=64)
    return _Cache(**{**f, **kw})


def strides():
    from kv_cached_qwen3_gb300.kv4 import _Strides
    return _Strides(0, 0, 128, 64)


BAD_CACHES = [dict(k=0), dict(v=0), dict(page_table=0), dict(k=4104), dict(n_pages=0), dict(n_streams=0),
              dict(pages_per_stream=0), dict(pages_per_stream=1 << 26), dict(n_layers=0), dict(n_kv_heads=-1),
              dict(head_dim=32), dict(head_dim=96)]


def test_page_bytes(lib):
    assert lib.talker_kv4_page_bytes(28, 8, 128) == 28 * 8 * 64 * (64 + 8)
    assert lib.talker_kv4_page_bytes(1, 1, 64) == 64 * (32 + 4)
    for bad in ((0, 1, 64), (1, 0, 64), (1, 1, 32), (1 << 20, 1 << 20, 128)):
        assert lib.talker_kv4_page_bytes(*bad) == 0


def test_rows_refusals(lib):
    st = strides()

    def call(c, layer0=0, n_layers=1, s0=0, n=1, T=1, k=256, v=512, dtype=0, st=ctypes.addressof(st)):
        ref_ = ctypes.addressof(c) if c is not None else None
        return [f(ref_, layer0, n_layers, s0, n, None, None, T, k, v, dtype, st, None)
                for f in (lib.talker_kv4_write, lib.talker_kv4_read)]
    good = cache()
    assert call(None) == [1, 1]
    for kw in BAD_CACHES:
        assert call(cache(**kw)) == [1, 1], kw
    for kw in (dict(k=0), dict(v=0), dict(st=None), dict(T=-1), dict(dtype=2), dict(dtype=3), dict(k=258), dict(layer0=3),
               dict(layer0=-1), dict(n_layers=4), dict(n_layers=-1), dict(s0=4), dict(n=5), dict(s0=-1), dict(T=1 << 30)):
        assert call(good, **kw) == [1, 1], kw
    for kw in (dict(T=0), dict(n=0), dict(n_layers=0)):           # nothing to do
        assert call(good, **kw) == [0, 0], kw


def test_attend_refusals(lib):
    def call(c, layer=0, B=1, lens=64, max_len=10, n_q=4, q=256, kn=None, vn=None, dtype=0, out=512, scratch=None, n=0):
        return lib.talker_kv4_attend(ctypes.addressof(c), layer, B, lens, max_len, n_q, 1.0, q, 0, kn, vn, 0, dtype, out,
                                     scratch, n, None)
    for kw in BAD_CACHES:
        assert call(cache(**kw)) == 1, kw
    for kw in (dict(layer=3), dict(layer=-1), dict(B=5), dict(B=-1), dict(lens=None), dict(max_len=-1), dict(n_q=3),
               dict(n_q=18), dict(n_q=0), dict(q=None), dict(out=None), dict(kn=256), dict(vn=256), dict(dtype=2),
               dict(q=257), dict(out=514), dict(q=257, dtype=1)):
        assert call(cache(), **kw) == 1, kw
    # a launch that needs scratch is refused without enough of it
    c = cache()
    need = lib.talker_kv4_attend_scratch(ctypes.addressof(c), 1, 4, 128)
    if need:
        for kw in (dict(scratch=None, n=need), dict(scratch=4096, n=need - 1), dict(scratch=4100, n=need)):
            assert call(c, max_len=128, **kw) == 1, kw
    assert lib.talker_kv4_attend_scratch(ctypes.addressof(c), 9, 4, 128) == 0
    assert call(c, B=0) == 0


def test_reorder_refusals(lib):
    def call(c, parents=1 << 20, R=4, lens=2 << 20, table=3 << 20, out=4 << 20):
        return lib.talker_kv4_reorder(ctypes.addressof(c), parents, R, lens, table, out, None)
    for kw in BAD_CACHES:
        assert call(cache(**kw)) == 1, kw
    for kw in (dict(parents=None), dict(R=5), dict(R=-1), dict(lens=None), dict(table=None), dict(out=None), dict(table=64),
               dict(table=92), dict(out=(2 << 20) + 4), dict(out=(3 << 20) + 16), dict(table=(1 << 20) + 12)):
        assert call(cache(), **kw) == 1, kw
    assert call(cache(n_pages=7)) == 1
    assert call(cache(n_streams=1025, n_pages=1 << 20)) == 1


def test_beam_refusals(lib):
    def call(x=4096, stride=200000, dtype=0, scores=64, ended=None, S=1, W=4, V=100, eos=-1, tok=256, par=512, best=768,
             done=None, scratch=1024, n=1 << 20):
        return lib.talker_beam_select(x, stride, dtype, scores, ended, S, W, V, eos, tok, par, best, done, scratch, n, None)
    need = lib.talker_beam_scratch(1, 4, 200000)
    assert need > 0 and lib.talker_beam_scratch(1, 4, 100) == 0
    for kw in (dict(x=None), dict(scores=None), dict(tok=None), dict(par=None), dict(best=None), dict(stride=99),
               dict(dtype=2), dict(W=0), dict(W=33), dict(V=3), dict(S=-1), dict(eos=100), dict(ended=64, eos=-1),
               dict(best=64), dict(ended=64, done=64, eos=1), dict(V=200000, scratch=None), dict(V=200000, scratch=1032),
               dict(V=200000, n=need - 1), dict(x=4098)):
        assert call(**kw) == 1, kw
    assert call(S=0) == 0
    for bad in ((-1, 4, 100), (1, 0, 100), (1, 33, 100), (1, 4, 3), (1 << 30, 4, 100), (1, 4, (1 << 30) + 1)):
        assert lib.talker_beam_scratch(*bad) == 0


def test_quantizer_definition():
    """Hand cases: borders go to the higher code, the first of +m and -m decides, a maximum of either sign is exact
    up to its scale's rounding."""
    x = np.zeros((1, 32))
    x[0, :6] = [8, -8, 0.5, -0.5, 7.5, 7.4]
    codes, d = ref.q4_quantize(x)
    assert d[0, 0] == -1.0
    # 8.5 - x: 0.5, 16.5, 8.0, 9.0, 1.0, 1.1, 8.5 ...
    assert codes[0, :7].tolist() == [0, 15, 8, 9, 1, 1, 8]
    assert ref.q4_values(codes, d)[0, :6].tolist() == [8, -7, 0, -1, 7, 7]
    codes, d = ref.q4_quantize(-x)
    assert d[0, 0] == 1.0 and codes[0, :7].tolist() == [0, 15, 8, 9, 1, 1, 8]
    codes, d = ref.q4_quantize(np.zeros((1, 32)))
    assert (codes == 8).all() and d[0, 0] == 0
    rng = np.random.default_rng(0)
    y = rng.standard_normal((100, 64))
    codes, d = ref.q4_quantize(y)
    assert codes.max() <= 15
    back = ref.q4_values(codes, d)
    m = np.abs(y.reshape(100, 2, 32)).max(-1)
    # half a step of |m| / 8, a whole one at the far end, and the scale's own rounding
    assert (np.abs(back - y).reshape(100, 2, 32).max(-1) <= m / 8 * (1 + 8 * 2.0 ** -11)).all()


def test_layout_round_trip():
    """tile_bytes places every dim of a row at a nibble of its own."""
    for hd in (64, 128):
        for is_v in (False, True):
            seen = set()
            for dim in range(hd):
                codes = np.zeros((64, hd), np.uint8)
                codes[5, dim] = 15
                t = ref.tile_bytes(codes, np.zeros((64, hd // 32)), is_v)
                at = np.flatnonzero(t)
                assert len(at) == 1 and 5 * hd // 2 <= at[0] < 6 * hd // 2
                seen.add((int(at[0]), int(t[at[0]])))
            assert len(seen) == hd
