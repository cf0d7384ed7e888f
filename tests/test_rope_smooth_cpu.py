"""CPU: frequencies scaled by wavelength, over every range of turns that the header allows."""
import ctypes
import math

import numpy as np
import pytest

import layer_ref as ref


@pytest.mark.parametrize("low,high", [(0.0, 4.0), (-1.0, 0.5), (1.0, 4.0), (-3.0, -1.0)])
def test_ranges_of_turns(low, high):
    from kv_cached_qwen3_gb300 import build, talker
    from kv_cached_qwen3_gb300.rotary import make_rope
    build.build()
    scaling = dict(type="smooth", factor=4.0, original=4096.0, low=low, high=high)
    turns, amp = np.zeros(32, np.uint64), ctypes.c_float()
    rope = make_rope(64, 1e4, scaling)
    assert talker.load_library().talker_rope_turns(ctypes.byref(rope), turns.ctypes.data, ctypes.byref(amp)) == 0
    want, _ = ref.frequencies(64, 1e4, scaling)
    # a few roundings of f64, and half of the table's step, 2^-65 turn, in radians
    assert (np.abs(turns.astype(np.float64) * 2.0 ** -64 * 2 * math.pi - want) <= want * 2.0 ** -46 + math.pi * 2.0 ** -64).all()
    assert amp.value == 1.0


@pytest.mark.parametrize("kind,low,high", [("smooth", 4.0, 4.0), ("smooth", math.nan, 4.0), ("smooth", -math.inf, 4.0), ("smooth", 1.0, math.inf),
                                           ("yarn", 0.0, 4.0), ("yarn", -1.0, 4.0), ("yarn", math.nan, 4.0)])
def test_refusals(kind, low, high):
    from kv_cached_qwen3_gb300 import build, talker
    from kv_cached_qwen3_gb300.rotary import _Rope, SCALINGS
    build.build()
    turns, amp = np.zeros(32, np.uint64), ctypes.c_float()
    rope = _Rope(64, SCALINGS[kind], 1e4, 4.0, 4096.0, low, high, 0.0)
    assert talker.load_library().talker_rope_turns(ctypes.byref(rope), turns.ctypes.data, ctypes.byref(amp)) == 1
