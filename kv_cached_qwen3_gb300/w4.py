"""Products with 4-bit weights in groups (include/talker_layer.h, talker_w4_*)."""
from __future__ import annotations

import ctypes

import torch

from .kv4 import _DTYPE, contiguous_rows, launch
from .norm import ROW_TYPES
from .talker import load_library


class _W4(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_void_p)] + [(n, ctypes.c_int32) for n in ("n", "k", "group", "zeros", "gated")]


def quantize(w, group: int = 32):
    """(codes, scales) of a dense matrix w [n, k], f32 or bf16 with contiguous rows: uint8 [n, ceil(k / 2)], two codes a byte
    (the even input in the low four bits), and fp16 [n, ceil(k / group)], by the rule of the 4-bit cache over groups of 32,
    64 or 128 inputs: a code c stands for (c - 8) scale."""
    dtype = _DTYPE.get(w.dtype)
    if w.dim() != 2 or dtype is None or not w.is_cuda or not contiguous_rows(w) or 0 in w.shape:
        raise ValueError("quantize: w must be an f32 or bf16 CUDA tensor [n, k] with contiguous rows")
    if group not in (32, 64, 128):
        raise ValueError("quantize: group must be 32, 64 or 128")
    n, k = w.shape
    codes = torch.empty(n, (k + 1) // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(n, -(-k // group), dtype=torch.float16, device=w.device)
    launch(w.device.index, load_library().talker_w4_quantize, "talker_w4_quantize", w.data_ptr(), dtype, w.stride(0), n, k, group,
           codes.data_ptr(), scales.data_ptr())
    return codes, scales


class W4Matrix:
    """A matrix [n, k] of 4-bit codes as the kernels read it, or two of them joined for silu(W x) * (U x)."""

    @classmethod
    def pack(cls, codes, scales, zeros=None, *, k: int, group: int, gated_with=None) -> "W4Matrix":
        """From codes uint8 [n, ceil(k / 2)], scales fp16 [n, ceil(k / group)] and zeros uint8 of the scales' shape (0..15; None: 8):
        the code c stands for (c - zero) scale. gated_with: (codes, scales[, zeros]) of U, of the same sizes."""
        self = cls.__new__(cls)
        if group not in (32, 64, 128) or k < 1:
            raise ValueError("W4Matrix: needs inputs, and groups of 32, 64 or 128")
        n, device = codes.shape[0], codes.device
        both = [(codes, scales, zeros)]
        if gated_with is not None:
            both.append(tuple(gated_with) + (None,) * (3 - len(gated_with)))
            if (both[1][2] is None) != (zeros is None):
                raise ValueError("W4Matrix: both matrices of a gated one have zeros, or none has")
        for c, s, z in both:
            for name, t, dt, shape in (("codes", c, torch.uint8, (n, (k + 1) // 2)), ("scales", s, torch.float16, (n, -(-k // group))),
                                       ("zeros", z, torch.uint8, (n, -(-k // group)))):
                if t is None and name == "zeros":
                    continue
                if t.shape != shape or t.dtype is not dt or t.device != device or not t.is_contiguous() or not t.is_cuda:
                    raise ValueError("W4Matrix: %s must be a contiguous %s CUDA tensor %s" % (name, dt, list(shape)))
        lib = load_library()
        self.n, self.k, self.group, self.gated, self.device = n, k, group, gated_with is not None, device
        self._c = _W4(0, n, k, group, zeros is not None, self.gated)
        self._ref = ctypes.addressof(self._c)
        size = lib.talker_w4_bytes(self._ref)
        if size == 0:
            raise ValueError("W4Matrix: sizes that are not supported")
        self.tiles = torch.empty(size, dtype=torch.uint8, device=device)
        self._c.tiles = self.tiles.data_ptr()
        at = [[None if t is None else t.data_ptr() for t in m] for m in both]
        launch(device.index, lib.talker_w4_pack, "talker_w4_pack", self._ref, *at[0], *(at[1] if self.gated else (None,) * 3))
        self._matmul, self._need, self._scratch = lib.talker_w4_matmul, lib.talker_w4_scratch, {}
        return self

    @classmethod
    def quantize(cls, w, group: int = 32, gated_with=None) -> "W4Matrix":
        """From a dense matrix (and U, of the same sizes): see quantize()."""
        other = None if gated_with is None else quantize(gated_with, group)
        if other is not None and gated_with.shape != w.shape:
            raise ValueError("W4Matrix: the matrices of a gated one have the same sizes")
        return cls.pack(*quantize(w, group), k=w.shape[1], group=group, gated_with=other)

    def matmul(self, x, x_scales=None, residual=None, out_dtype=None, out=None):
        """W x for rows x [rows, k]: f32, bf16, or float8_e4m3fn with x_scales f32 [rows, blocks] as rms_norm gives them. Of a
        gated matrix silu(W x) * (U x). residual [rows, n] in the result's type is added. Returns [rows, n] f32 or bf16
        (out_dtype; default x's type, of 8-bit rows f32); out names a tensor to write to, which may be residual."""
        xt, shape = ROW_TYPES.get(x.dtype), x.shape
        if len(shape) != 2 or xt is None or shape[1] != self.k or x.device != self.device or not contiguous_rows(x):
            raise ValueError("matmul: x must be f32, bf16 or float8_e4m3fn [rows, %d] on %s with contiguous rows" % (self.k, self.device))
        rows, block = shape[0], 0
        if xt == 4:
            blocks = 0 if x_scales is None or x_scales.dim() != 2 else x_scales.shape[1]
            block = 0 if blocks == 1 else next((b for b in (32, 64, 128) if -(-self.k // b) == blocks), None)
            if block is None or x_scales is None or x_scales.shape[0] != rows or x_scales.dtype is not torch.float32 or \
                    x_scales.device != self.device or not x_scales.is_contiguous():
                raise ValueError("matmul: x_scales must be contiguous f32 [rows, 1] or [rows, ceil(k / 32, 64 or 128)]")
        elif x_scales is not None:
            raise ValueError("matmul: x_scales go with float8_e4m3fn rows")
        if out_dtype is None:
            out_dtype = out.dtype if out is not None else torch.float32 if xt == 4 else x.dtype
        ot = _DTYPE.get(out_dtype)
        if ot is None:
            raise ValueError("matmul: out_dtype must be float32 or bfloat16")
        if out is None:
            out = torch.empty((rows, self.n), dtype=out_dtype, device=self.device)
        elif out.shape != (rows, self.n) or out.dtype is not out_dtype or out.device != self.device or not contiguous_rows(out):
            raise ValueError("matmul: out must be [rows, %d] with contiguous rows" % self.n)
        if residual is not None and (residual.shape != out.shape or residual.dtype is not out_dtype or
                                     residual.device != self.device or not contiguous_rows(residual)):
            raise ValueError("matmul: residual must be [rows, %d] in the result's type with contiguous rows" % self.n)
        if rows == 0:
            return out
        need = self._scratch.get((xt, rows))
        if need is None:
            if len(self._scratch) >= 256:
                self._scratch.clear()
            need = self._scratch[(xt, rows)] = self._need(self._ref, xt, rows)
        scratch = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        launch(self.device.index, self._matmul, "talker_w4_matmul", self._ref, x.data_ptr(), xt, x.stride(0),
               None if x_scales is None else x_scales.data_ptr(), block, rows, None if residual is None else residual.data_ptr(),
               0 if residual is None else residual.stride(0), out.data_ptr(), ot, out.stride(0),
               scratch.data_ptr() if need else None, need)
        return out
