"""CPU: results whose rows or heads would be written to one place are refused before anything is enqueued. (Their inputs may lie
so: a residual or a position's heads that all rows share.)"""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from kv_cached_qwen3_gb300 import build, talker
    build.build()
    return talker.load_library()


def test_norm(lib):
    from kv_cached_qwen3_gb300.norm import _RowStrides

    def call(rows, inner, s=(192, 64), y=(192, 64)):
        at = [_RowStrides(*v) for v in ((0, 0), (0, 0), s, y)]
        x, r, so, yo = map(ctypes.addressof, at)
        return lib.talker_rms_norm(256, 0, x, 512, 0, r, 1024, 1e-6, rows, inner, 64, 2048, so, 4096, 0, yo, 0, None, None)
    for kw in (dict(rows=2, inner=1, y=(0, 64)), dict(rows=2, inner=1, s=(0, 64)), dict(rows=6, inner=3, y=(0, 64)), dict(rows=6, inner=3, y=(192, 0)),
               dict(rows=6, inner=3, s=(192, 0)), dict(rows=2, inner=3, s=(192, 0)), dict(rows=2, inner=3, y=(0, 0))):
        assert call(**kw) == 1, kw


def test_rotate(lib):
    from kv_cached_qwen3_gb300.rotary import _Heads

    def call(streams, rows, heads, second=False, **kw):
        good = dict(at=1024, out=1024, heads=heads, in_stream=0, in_row=0, in_head=0, out_stream=4096, out_row=256, out_head=64)
        sets = (_Heads * 2)(_Heads(**(good if second else {**good, **kw})), _Heads(**{**good, **kw}))
        return lib.talker_rotate(256, 1.0, 64, 64, 0, 512, streams, rows, ctypes.addressof(sets), 2 if second else 1, 0, None)
    for second in (False, True):
        for kw in (dict(out_stream=0), dict(out_row=0), dict(out_head=0)):
            assert call(2, 3, 4, second, **kw) == 1, kw
