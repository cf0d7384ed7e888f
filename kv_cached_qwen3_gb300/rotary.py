"""Rotary positions (include/talker_layer.h, talker_rotate)."""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from .kv4 import _DTYPE, launch
from .talker import TalkerError, load_library

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "smooth": 3, "yarn": 4}


class _Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32)] + [(n, ctypes.c_double) for n in (
        "theta", "factor", "original", "low", "high", "amplitude")]


class _Heads(ctypes.Structure):
    _fields_ = [("at", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int32)] + [
        (n, ctypes.c_int64) for n in ("in_stream", "in_row", "in_head", "out_stream", "out_row", "out_head")]


def make_rope(rotary_dim: int, theta: float, scaling: dict | None) -> _Rope:
    """The C struct of a rope with a scaling as Rotary describes it."""
    given = dict(scaling or {"type": "none"})
    kind = given.pop("type", None)
    names = {"none": (), "linear": ("factor",), "ntk": ("factor",), "smooth": ("factor", "original", "low", "high"),
             "yarn": ("factor", "original", "beta_slow", "beta_fast")}.get(kind)
    if names is None or not set(names) <= set(given) or set(given) - set(names) - ({"amplitude"} if kind == "yarn" else set()):
        raise ValueError("rotary positions: scaling %r" % (scaling,))
    v = [float(given[n]) for n in names]
    return _Rope(rotary_dim, SCALINGS[kind], theta, *(v + [0.0] * (4 - len(v))), float(given.get("amplitude", 0.0)))


class Rotary:
    """The plan of a rope: its table of frequencies on a device.

    scaling: None, or a dict with "type" and its numbers:
      {"type": "linear", "factor"}, {"type": "ntk", "factor"},
      {"type": "smooth", "factor", "original", "low", "high"}
      {"type": "yarn", "factor", "original", "beta_fast", "beta_slow", "amplitude" (absent: by the factor)}
    where `original` counts the positions of the context that the frequencies were trained for."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None, theta: float = 1e6, interleaved: bool = False,
                 scaling: dict | None = None, device="cuda"):
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if not 2 <= head_dim <= 512 or rotary_dim < 2 or rotary_dim % 2 or rotary_dim > head_dim:
            raise ValueError("Rotary: needs head_dim 2 to 512 and an even rotary_dim of at most head_dim")
        if torch.device(device).type != "cuda":
            raise ValueError("Rotary: needs a CUDA device")
        rope = make_rope(rotary_dim, theta, scaling)
        table = np.empty(rotary_dim // 2, np.uint64)
        amplitude = ctypes.c_float()
        lib = load_library()
        st = lib.talker_rope_turns(ctypes.byref(rope), table.ctypes.data, ctypes.byref(amplitude))
        if st != 0:
            raise TalkerError(st, "talker_rope_turns")
        self.head_dim, self.rotary_dim, self.interleaved = head_dim, rotary_dim, bool(interleaved)
        self.amplitude = amplitude.value
        self.turns = torch.from_numpy(table.view(np.int64)).to(device)
        self.device = self.turns.device
        self._rotate = lib.talker_rotate

    def rotate(self, q, k, positions, out=None):
        """(q, k) with their heads turned to their rows' positions. q, and k unless it is None: f32 or bf16 [rows, heads,
        head_dim] with positions [rows], or [streams, rows, heads, head_dim] with positions [streams, rows], in any
        strides with contiguous dims; positions contiguous int32, any value. out: a pair of tensors to write to,
        which may be (q, k) themselves."""
        dims, device, dtype = q.dim(), self.device, _DTYPE.get(q.dtype)
        if dtype is None or dims not in (3, 4) or (k is not None and k.dtype is not q.dtype):
            raise ValueError("rotate: q and k must be f32 or bf16 [rows, heads, %d] or [streams, rows, heads, %d]" %
                             (self.head_dim, self.head_dim))
        rows = q.shape[:dims - 2]
        if positions.shape != rows or positions.dtype is not torch.int32 or positions.device != device or \
                not positions.is_contiguous():
            raise ValueError("rotate: positions must be contiguous int32 %s on %s" % (list(rows), device))
        sets, new = (_Heads * 2)(), []
        n = 1 if k is None else 2
        for i in range(n):
            t = k if i else q
            shape, s = t.shape, t.stride()
            if len(shape) != dims or shape[:dims - 2] != rows or shape[-1] != self.head_dim or t.device != device or s[-1] != 1:
                raise ValueError("rotate: q and k must have the same rows, head_dim %d with contiguous dims, and device %s" %
                                 (self.head_dim, device))
            if out is None:
                o = torch.empty(shape, dtype=q.dtype, device=device)
            else:
                o = out[i]
                if o.shape != shape or o.dtype is not q.dtype or o.device != device or o.stride(-1) != 1:
                    raise ValueError("rotate: out must be tensors of q's and k's shapes and type with contiguous dims")
            new.append(o)
            u = o.stride()
            if t.numel():
                h = sets[i]
                h.at, h.out, h.heads = t.data_ptr(), o.data_ptr(), shape[-2]
                h.in_row, h.in_head, h.out_row, h.out_head = s[-3], s[-2], u[-3], u[-2]
                if dims == 4:
                    h.in_stream, h.out_stream = s[0], u[0]
            else:
                h = sets[i]
                h.at, h.out = self.turns.data_ptr(), self.turns.data_ptr()     # (no heads: not read)
        if 0 not in rows:
            launch(device.index, self._rotate, "talker_rotate", self.turns.data_ptr(), self.amplitude, self.head_dim,
                   self.rotary_dim, self.interleaved, positions.data_ptr(), rows[0] if dims == 4 else 1, rows[-1],
                   ctypes.addressof(sets), n, dtype)
        return (new[0], new[1] if n == 2 else None)
