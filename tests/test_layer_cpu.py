"""CPU: what the layer operators and the drafts' verification refuse before they touch a GPU, and the host's tables."""
import ctypes
import math

import numpy as np
import pytest

import layer_ref as ref


@pytest.fixture(scope="module")
def lib():
    from kv_cached_qwen3_gb300 import build, talker
    build.build()
    return talker.load_library()


def test_norm_refusals(lib):
    from kv_cached_qwen3_gb300.norm import _RowStrides
    st = _RowStrides(64, 0)
    at = ctypes.addressof(st)

    def call(x=256, xt=0, xs=at, res=512, rt=1, rs=at, gain=1024, eps=1e-6, rows=1, inner=1, width=64, s=2048, ss=at, y=4096, yt=4,
             ys=at, block=32, scales=8192):
        return lib.talker_rms_norm(x, xt, xs, res, rt, rs, gain, eps, rows, inner, width, s, ss, y, yt, ys, block, scales, None)
    assert call(rows=0) == 0
    for kw in (dict(x=None), dict(x=257), dict(x=258), dict(xt=2), dict(xt=4), dict(xs=None), dict(rt=4), dict(rt=2), dict(rs=None), dict(res=513),
               dict(res=None), dict(gain=None), dict(gain=1026), dict(eps=-1.0), dict(eps=math.nan), dict(rows=-1), dict(rows=(1 << 30) + 1),
               dict(inner=0), dict(width=0), dict(width=(1 << 24) + 1), dict(ss=None), dict(s=2049), dict(y=None), dict(yt=3), dict(ys=None),
               dict(block=16), dict(block=-1), dict(block=256), dict(scales=None), dict(scales=8194), dict(yt=0, y=4098)):
        assert call(**kw) == 1, kw


def test_rope_tables(lib):
    from kv_cached_qwen3_gb300.rotary import SCALINGS, _Rope

    def table(d, kind, theta=1e6, factor=4.0, original=4096.0, low=1.0, high=32.0, amplitude=0.0):
        turns, amp = np.zeros(max(1, d // 2), np.uint64), ctypes.c_float()
        r = _Rope(d, kind if isinstance(kind, int) else SCALINGS[kind], theta, factor, original, low, high, amplitude)
        return lib.talker_rope_turns(ctypes.byref(r), turns.ctypes.data, ctypes.byref(amp)), turns, amp.value
    given = {"none": None, "linear": dict(type="linear", factor=4.0), "ntk": dict(type="ntk", factor=4.0),
             "smooth": dict(type="smooth", factor=4.0, original=4096.0, low=1.0, high=32.0),
             "yarn": dict(type="yarn", factor=4.0, original=4096.0, beta_slow=1.0, beta_fast=32.0)}
    for kind, scaling in given.items():
        for d in (4, 64, 80, 128):
            for theta in (1e4, 1e6):
                st, turns, amp = table(d, kind, theta)
                want, wamp = ref.frequencies(d, theta, scaling)
                assert st == 0
                # a few roundings of f64 in f, and half of the table's step, 2^-65 turn, in radians: pi 2^-64
                got = turns.astype(np.float64) * 2.0 ** -64 * 2 * math.pi
                assert (np.abs(got - want) <= want * 2.0 ** -46 + math.pi * 2.0 ** -64).all()
                assert abs(amp - wamp) <= 2.0 ** -24 * wamp
    assert table(128, "yarn", amplitude=0.5)[2] == 0.5
    for kw in (dict(d=0), dict(d=7), dict(d=-2), dict(kind=5), dict(kind=-1), dict(theta=1.0), dict(theta=math.inf), dict(theta=math.nan), dict(factor=0.5),
               dict(factor=math.nan), dict(original=0.0), dict(low=0.0), dict(low=32.0), dict(high=math.inf), dict(amplitude=-1.0), dict(d=2, kind="ntk")):
        assert table(**{**dict(d=64, kind="yarn"), **kw})[0] == 1, kw
    assert lib.talker_rope_turns(None, None, None) == 1


def test_rotate_refusals(lib):
    from kv_cached_qwen3_gb300.rotary import _Heads

    def call(turns=256, hd=64, rd=64, pos=512, streams=1, rows=1, n=1, dtype=0, null=False, **kw):
        sets = (_Heads * 2)(_Heads(**{**dict(at=1024, out=1024, heads=2, in_row=128, in_head=64, out_row=128, out_head=64), **kw}))
        return lib.talker_rotate(turns, 1.0, hd, rd, 0, pos, streams, rows, None if null else ctypes.addressof(sets), n, dtype, None)
    for kw in (dict(rows=0), dict(streams=0), dict(heads=0)):
        assert call(**kw) == 0, kw
    for kw in (dict(turns=None), dict(turns=260), dict(pos=None), dict(pos=513), dict(hd=1), dict(hd=513), dict(rd=0), dict(rd=63), dict(rd=66), dict(streams=-1), dict(rows=-1),
               dict(n=0), dict(n=3), dict(dtype=2), dict(at=None), dict(out=None), dict(heads=-1), dict(heads=16385), dict(streams=1 << 16, rows=1 << 15), dict(at=1026), dict(out=1025, dtype=1),
               dict(null=True), dict(n=2)):
        assert call(**kw) == 1, kw


def matrix(**kw):
    from kv_cached_qwen3_gb300.w4 import _W4
    return _W4(**{**dict(tiles=4096, n=33, k=130, group=64, zeros=1, gated=0), **kw})


BAD_MATRICES = [dict(n=0), dict(n=-1), dict(n=(1 << 27) + 1), dict(k=0), dict(k=(1 << 20) + 1), dict(group=16), dict(group=0), dict(group=256), dict(zeros=2), dict(gated=-1)]


def test_w4_refusals(lib):
    def r(c):
        return None if c is None else ctypes.addressof(c)
    good = matrix()
    assert lib.talker_w4_bytes(r(good)) == 3 * 2 * (1024 + 64 + 32)
    assert lib.talker_w4_bytes(r(matrix(gated=1, zeros=0))) == 5 * 2 * (1024 + 64)
    assert lib.talker_w4_bytes(r(matrix(group=128))) == 3 * 2 * (1024 + 32 + 32)
    assert lib.talker_w4_bytes(None) == 0

    def pack(c, codes=64, scales=128, zeros=192, codes2=256, scales2=320, zeros2=384):
        return lib.talker_w4_pack(r(c), codes, scales, zeros, codes2, scales2, zeros2, None)

    def matmul(c, x=64, xt=0, x_row=130, xs=None, block=0, rows=2, res=None, res_row=33, out=512, ot=0, out_row=33, scratch=1024, need=1 << 30):
        return lib.talker_w4_matmul(r(c), x, xt, x_row, xs, block, rows, res, res_row, out, ot, out_row, scratch, need, None)
    for kw in BAD_MATRICES:
        c = matrix(**kw)
        assert lib.talker_w4_bytes(r(c)) == 0 and pack(c) == 1 and matmul(c) == 1 and lib.talker_w4_scratch(r(c), 0, 1) == 0, kw
    for c in (None, matrix(tiles=None), matrix(tiles=4104)):
        assert pack(c) == 1 and matmul(c) == 1
    for kw in (dict(codes=None), dict(scales=None), dict(scales=129), dict(zeros=None)):
        assert pack(good, **kw) == 1, kw
    for kw in (dict(codes2=None), dict(scales2=None), dict(scales2=321), dict(zeros2=None)):
        assert pack(matrix(gated=1), **kw) == 1, kw
    assert matmul(good, rows=0) == 0
    for kw in (dict(x=None), dict(x=66), dict(xt=2), dict(xt=3), dict(xt=4), dict(xt=4, xs=130), dict(xt=4, xs=128, block=16), dict(rows=-1), dict(rows=(1 << 16) + 1),
               dict(out=None), dict(out=513), dict(ot=4), dict(out_row=32), dict(res=514), dict(res=512, res_row=40), dict(need=1), dict(scratch=1032), dict(scratch=None)):
        assert matmul(good, **kw) == 1, kw

    def quantize(w=64, dtype=0, stride=130, n=4, k=130, group=32, codes=128, scales=256):
        return lib.talker_w4_quantize(w, dtype, stride, n, k, group, codes, scales, None)
    for kw in (dict(w=None), dict(w=65), dict(dtype=2), dict(stride=129), dict(n=0), dict(k=0), dict(group=48), dict(codes=None), dict(scales=None), dict(scales=257)):
        assert quantize(**kw) == 1, kw


def test_draft_refusals(lib):
    def call(t=64, ts=30, tr=10, d=128, ds=20, dr=10, dtype=0, tok=256, cnt=None, u=320, temp=None, S=1, K=2, V=10, out=384, acc=448, lp=512, scratch=1024, need=1 << 30):
        return lib.talker_draft_verify(t, ts, tr, d, ds, dr, dtype, tok, cnt, u, temp, S, K, V, out, acc, lp, scratch, need, None)
    assert call(S=0) == 0
    for kw in (dict(t=None), dict(t=66), dict(d=130), dict(t=65, dtype=1), dict(dtype=2), dict(dtype=4), dict(tok=None), dict(u=None), dict(S=-1), dict(S=65536), dict(K=-1), dict(K=65),
               dict(V=0), dict(V=(1 << 26) + 1), dict(out=None), dict(acc=None), dict(tok=257), dict(cnt=66), dict(u=322), dict(temp=513), dict(out=386),
               dict(acc=449), dict(lp=514)):
        assert call(**kw) == 1, kw


def test_draft_reference_on_hand_cases():
    """The tests' own definition: a refused draft's token comes from what is left of p, a certain draft leaves p without its token."""
    t = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.2, 0.7]]))
    d = np.log(np.array([[0.2, 0.7, 0.1]]))
    # u q(1) = 0.35 is not below 0.25: refused; what is left: .3, 0, .15 -> border at 0.3 / 0.45
    assert ref.verify(t, [1], [0.5, 0.66], d)[:2] == ([0, -1], 0)
    assert ref.verify(t, [1], [0.5, 0.67], d)[:2] == ([2, -1], 0)
    assert ref.verify(t, [1], [0.35, 0.05], d)[:2] == ([1, 0], 1)
    assert ref.verify(t, [0], [0.6, 0.4])[:2] == ([1, -1], 0)
    assert ref.verify(t, [2], [0.2, 0.31])[:2] == ([2, 2], 1)
    assert ref.verify(t, [1], [0.0, 0.5], temp=0.0)[:2] == ([0, -1], 0)
    assert ref.verify(t, [0], [0.0, 0.5], temp=0.0)[:2] == ([0, 2], 1)


def test_rope_scaling_of_a_talker_refusals(lib):
    assert lib.talker_set_rope_scaling(None, None) == 1
