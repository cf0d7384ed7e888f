"""Residual addition and RMSNorm (include/talker_layer.h, talker_rms_norm)."""
from __future__ import annotations

import ctypes

import torch

from .kv4 import contiguous_rows, launch
from .talker import load_library

ROW_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 4}


class _RowStrides(ctypes.Structure):
    _fields_ = [("outer", ctypes.c_int64), ("inner", ctypes.c_int64)]


_strides = {}     # structs by their values: calls of a program have few


def _at(t, dims):
    """(address, struct) of a _RowStrides for rows of t (2 or 3 dims, or more that are contiguous). The pair is what keeps the
    struct: whoever hands the address on holds it until the library has returned, for the table may have let go of it."""
    s = t.stride()
    key = (s[0], 0) if dims == 2 else (s[0], s[1]) if dims == 3 else (t.shape[-1], 0)
    found = _strides.get(key)
    if found is None:
        if len(_strides) >= 4096:
            _strides.clear()
        struct = _RowStrides(*key)
        found = _strides[key] = (ctypes.addressof(struct), struct)
    return found


def rms_norm(x, gain, eps: float = 1e-6, residual=None, out_dtype=None, block: int = 0, out=None, sum_out=None):
    """(y, s, scales) of s = x + residual (s = x without one) and y = s / sqrt(mean(s^2) + eps) * gain.

    x, residual: f32 or bf16 [rows, width], or [rows, heads, width] in any strides with contiguous values (more dims
    where they are contiguous); gain f32 [width]. The norm is that of the f32 sum; s comes back in residual's type
    (None without a residual). y has out_dtype (default: x's): f32, bf16, or float8_e4m3fn, where blocks of `block` values
    (32, 64 or 128; 0: the whole row) share an f32 scale max|y| / 448 and y stands for codes * scales; scales is
    [..., ceil(width / block)], else None. out and sum_out name tensors to write to; sum_out may be residual or x
    itself, and out x or residual."""
    shape, device = x.shape, x.device
    dims = len(shape)
    xt = ROW_TYPES.get(x.dtype, 4)
    if dims < 2 or xt == 4 or device.type != "cuda" or not contiguous_rows(x) or shape[-1] < 1:
        raise ValueError("rms_norm: x must be an f32 or bf16 CUDA tensor [..., width] with contiguous values")
    width = shape[-1]
    rows = x.numel() // width
    if gain.dtype is not torch.float32 or gain.numel() != width or not gain.is_contiguous() or gain.device != device:
        raise ValueError("rms_norm: gain must be contiguous f32 [%d] on %s" % (width, device))
    out_dtype = x.dtype if out_dtype is None else out_dtype
    yt = ROW_TYPES.get(out_dtype)
    if yt is None:
        raise ValueError("rms_norm: out_dtype must be float32, bfloat16 or float8_e4m3fn")
    if block not in (0, 32, 64, 128):
        raise ValueError("rms_norm: block must be 0, 32, 64 or 128")
    if residual is None:
        if sum_out is not None:
            raise ValueError("rms_norm: sum_out needs a residual")
        rt, s = 0, None
    else:
        rt = ROW_TYPES.get(residual.dtype, 4)
        if residual.shape != shape or rt == 4 or residual.device != device or not contiguous_rows(residual):
            raise ValueError("rms_norm: residual must be f32 or bf16 of x's shape and device with contiguous values")
        s = torch.empty(shape, dtype=residual.dtype, device=device) if sum_out is None else sum_out
        if sum_out is not None and (s.shape != shape or s.dtype is not residual.dtype or s.device != device or not contiguous_rows(s)):
            raise ValueError("rms_norm: sum_out must have residual's shape and type and contiguous values")
    if out is None:
        y = torch.empty(shape, dtype=out_dtype, device=device)
    else:
        y = out
        if y.shape != shape or y.dtype is not out_dtype or y.device != device or not contiguous_rows(y):
            raise ValueError("rms_norm: out must have x's shape, out_dtype and contiguous values")
    if dims > 3 and not all(t is None or t.is_contiguous() for t in (x, residual, s, y)):
        raise ValueError("rms_norm: tensors of more than 3 dims must be contiguous")
    scales = None
    if yt == 4:
        scales = torch.empty(shape[:-1] + (-(-width // block) if block else 1,), dtype=torch.float32, device=device)
    if rows == 0:
        return y, s, scales
    none = (None, None)
    x_at, y_at = _at(x, dims), _at(y, dims)
    r_at, s_at = (none, none) if residual is None else (_at(residual, dims), _at(s, dims))
    launch(device.index, load_library().talker_rms_norm, "talker_rms_norm", x.data_ptr(), xt, x_at[0],
           None if residual is None else residual.data_ptr(), rt, r_at[0], gain.data_ptr(), eps, rows,
           shape[1] if dims == 3 else 1, width, None if s is None else s.data_ptr(), s_at[0], y.data_ptr(), yt, y_at[0],
           block, None if scales is None else scales.data_ptr())
    return y, s, scales
