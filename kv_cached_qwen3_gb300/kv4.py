"""The 4-bit paged KV cache (include/talker_kv4.h): rows written, read back and attended, streams reordered.

PyTorch holds the memory and names the stream; every step runs in libtalker_gb300.so. Calls are
enqueued on the current stream of the cache's device and can be captured into CUDA graphs.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .talker import TalkerError, load_library

PAGE = 64
# torch.cuda.current_stream(device).cuda_stream and torch.cuda.current_device(), without their objects and checks:
# small calls take about as long as these (the tensors that are passed have initialised CUDA)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_DTYPE = {torch.float32: 0, torch.bfloat16: 1}


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("status", ctypes.c_void_p)] + [(n, ctypes.c_int32) for n in (
                    "n_pages", "n_streams", "pages_per_stream", "n_layers", "n_kv_heads", "head_dim")]


class _Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("layer", "stream", "row", "head")]


def launch(device: int, fn, what, *args):
    """fn(*args, stream) on the current stream of a device, with that device current."""
    if _current_device() == device:
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status != 0:
        raise TalkerError(status, what)


class KV4Cache:
    """Pools of 4-bit pages and the page table that names each stream's pages.

    k, v: uint8 [n_pages, n_layers, n_kv_heads, 36 * head_dim]; page_table: int32 [n_streams,
    pages_per_stream]; status: int32 [1], the word in which kernels report what only they can see.
    """

    def __init__(self, n_streams: int, max_seq_len: int, n_layers: int, n_kv_heads: int, head_dim: int, device="cuda"):
        if n_streams < 1 or max_seq_len < 1:
            raise ValueError("KV4Cache: n_streams and max_seq_len must be at least 1")
        if n_layers < 1 or n_kv_heads < 1 or head_dim not in (64, 128):
            raise ValueError("KV4Cache: needs layers, KV heads and head_dim 64 or 128")
        pps = (max_seq_len + PAGE - 1) // PAGE
        shape = (n_streams * pps, n_layers, n_kv_heads, 36 * head_dim)
        k = torch.zeros(shape, dtype=torch.uint8, device=device)
        table = torch.arange(n_streams * pps, dtype=torch.int32, device=device).view(n_streams, pps)
        self._init(k, torch.zeros_like(k), table, head_dim, None)

    @classmethod
    def over(cls, k, v, page_table, head_dim: int, status=None) -> "KV4Cache":
        """A cache over pools and a page table that the caller already has."""
        self = cls.__new__(cls)
        self._init(k, v, page_table, head_dim, status)
        return self

    def _init(self, k, v, page_table, head_dim, status):
        if head_dim not in (64, 128):
            raise ValueError("KV4Cache: head_dim must be 64 or 128")
        for name, t in (("k", k), ("v", v)):
            if t.dtype != torch.uint8 or t.dim() != 4 or t.shape[3] != 36 * head_dim or not t.is_contiguous() \
                    or not t.is_cuda:
                raise ValueError("KV4Cache: %s must be a contiguous uint8 CUDA tensor [n_pages, n_layers, n_kv_heads, "
                                 "%d]" % (name, 36 * head_dim))
        if k.shape != v.shape or k.device != v.device:
            raise ValueError("KV4Cache: k and v must have the same shape and device")
        self.k, self.v, self.head_dim, self.device = k, v, head_dim, k.device
        self.n_pages, self.n_layers, self.n_kv_heads = k.shape[:3]
        self._ints("page_table", page_table, None)
        if page_table.dim() != 2:
            raise ValueError("KV4Cache: page_table must be [n_streams, pages_per_stream]")
        self.page_table = page_table
        self.n_streams, self.pages_per_stream = page_table.shape
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._ints("status", status, 1)
        self.status = status
        self._lib = lib = load_library()
        self._write, self._read = lib.talker_kv4_write, lib.talker_kv4_read
        self._attend, self._reorder = lib.talker_kv4_attend, lib.talker_kv4_reorder
        self._c = _Cache(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), status.data_ptr(), self.n_pages,
                         self.n_streams, self.pages_per_stream, self.n_layers, self.n_kv_heads, head_dim)
        self._ref = ctypes.addressof(self._c)
        self._scratch = {}     # attend's scratch bytes by (B, n_q_heads, max_len)

    def _ints(self, name, t, n):
        if t.dtype is not torch.int32 or t.device != self.device or (n is not None and t.numel() != n) or \
                not t.is_contiguous():
            raise ValueError("%s must be a contiguous int32 tensor%s on %s" %
                             (name, "" if n is None else " of %d" % n, self.device))
        return t.data_ptr()

    def _rows(self, fn, what, k, v, start, count, layer0, stream0):
        shape, stride, dtype = k.shape, k.stride(), _DTYPE.get(k.dtype)
        if len(shape) != 5 or dtype is None or k.device != self.device or shape[3] != self.n_kv_heads or \
                shape[4] != self.head_dim:
            raise ValueError("%s: k and v must be f32 or bf16 [layers, streams, rows, %d, %d] on %s" %
                             (what, self.n_kv_heads, self.head_dim, self.device))
        if v.shape != shape or v.dtype is not k.dtype or v.device != self.device:
            raise ValueError("%s: k and v must have the same shape, type, strides and device" % what)
        if v.stride() != stride:      # (a dimension of one element has no stride)
            stride = tuple(a if n > 1 else 0 for n, a in zip(shape, stride))
            if stride != tuple(a if n > 1 else 0 for n, a in zip(shape, v.stride())):
                raise ValueError("%s: k and v must have the same shape, type, strides and device" % what)
        layers, streams, rows = shape[:3]
        if layers == 0 or streams == 0 or rows == 0:
            return
        if stride[4] != 1:
            raise ValueError("%s: the dims of k and v must be contiguous" % what)
        strides = _Strides(*stride[:4])
        launch(self.device.index, fn, what, self._ref, layer0, layers, stream0, streams,
               None if start is None else self._ints("start", start, streams),
               None if count is None else self._ints("count", count, streams), rows, k.data_ptr(), v.data_ptr(),
               dtype, ctypes.addressof(strides))

    def write(self, k, v, start=None, count=None, layer0: int = 0, stream0: int = 0):
        """Quantize rows into the cache. k, v: [layers, streams, rows, n_kv_heads, head_dim] f32 or bf16 in any
        strides with contiguous dims, for layers layer0.. and streams stream0..; row i of stream s goes to position
        start[s] + i (start None: 0), and rows past count[s] are not written."""
        self._rows(self._write, "talker_kv4_write", k, v, start, count, layer0, stream0)

    def read(self, k, v, start=None, count=None, layer0: int = 0, stream0: int = 0):
        """Read the rows that `write` with these arguments stores, into k and v, as the values they stand for. Rows
        past count[s] are left as they are. Returns (k, v)."""
        self._rows(self._read, "talker_kv4_read", k, v, start, count, layer0, stream0)
        return k, v

    def attend(self, layer: int, q, lens, k_new=None, v_new=None, scale=None, max_len=None, out=None):
        """softmax(scale q K^T) V for one query row per stream: q [B, n_q_heads, head_dim] f32 or bf16 (streams
        0..B-1), over the first lens[b] cached rows and, with k_new / v_new [B, n_kv_heads, head_dim], the step's own
        row as given. scale defaults to 1 / sqrt(head_dim); max_len is an estimate of the longest length (default:
        the streams' capacity) that shapes the launch. Returns [B, n_q_heads, head_dim] in q's type."""
        dtype = _DTYPE.get(q.dtype)
        shape = q.shape
        if len(shape) != 3 or dtype is None or q.device != self.device or shape[2] != self.head_dim:
            raise ValueError("attend: q must be f32 or bf16 [B, n_q_heads, %d] on %s" % (self.head_dim, self.device))
        B, n_q, hd = shape
        if n_q < 1 or n_q % self.n_kv_heads or n_q // self.n_kv_heads > 8 or B > self.n_streams:
            raise ValueError("attend: needs at most %d streams and 1 to 8 query heads per KV head" % self.n_streams)
        if (k_new is None) != (v_new is None):
            raise ValueError("attend: k_new and v_new go together")
        q = _dense_heads(q)
        kn = vn = None
        new_row = 0
        if k_new is not None:
            for t in (k_new, v_new):
                if t.shape != (B, self.n_kv_heads, hd) or t.dtype is not q.dtype or t.device != self.device:
                    raise ValueError("attend: k_new and v_new must be [B, n_kv_heads, head_dim] in q's type")
            k_new, v_new = _dense_heads(k_new), _dense_heads(v_new)
            if k_new.stride(0) != v_new.stride(0):
                k_new, v_new = k_new.contiguous(), v_new.contiguous()
            kn, vn, new_row = k_new.data_ptr(), v_new.data_ptr(), k_new.stride(0)
        lens_at = self._ints("lens", lens, B)
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=self.device)
        elif out.shape != shape or out.dtype is not q.dtype or out.device != self.device or not out.is_contiguous():
            raise ValueError("attend: out must be contiguous, with q's shape and type")
        if B == 0:
            return out
        if max_len is None:
            max_len = self.pages_per_stream * PAGE
        max_len = min(-(-max_len // PAGE), self.pages_per_stream) * PAGE      # whole pages: few different calls
        need = self._scratch.get((B, n_q, max_len))
        if need is None:
            with torch.cuda.device(self.device):      # (by its multiprocessors)
                need = self._scratch[(B, n_q, max_len)] = self._lib.talker_kv4_attend_scratch(self._ref, B, n_q, max_len)
        scratch = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        launch(self.device.index, self._attend, "talker_kv4_attend", self._ref, layer, B, lens_at, max_len, n_q,
               1.0 / math.sqrt(hd) if scale is None else scale, q.data_ptr(), q.stride(0), kn, vn, new_row,
               dtype, out.data_ptr(), scratch.data_ptr() if need else None, need)
        return out

    def reorder(self, parents, lens, table_out=None, lens_out=None):
        """Beam reordering: returns (cache, lens) in which stream i holds what stream parents[i] holds here under
        lens. Pools are shared: full pages are named by several streams, and only rows of a page that is still being
        filled are copied. This cache must not be used after rows are written through the new one. Streams that share
        pages and are cut (a smaller lens) get pages of their own to write to by a call without parents (a tensor of 0)."""
        R = parents.numel()
        at = self._ints("parents", parents, R)
        lens_at = self._ints("lens", lens, self.n_streams)
        if table_out is None:
            table_out = torch.empty_like(self.page_table)
            table_at = table_out.data_ptr()
        elif table_out.shape != self.page_table.shape:
            raise ValueError("reorder: table_out must be [n_streams, pages_per_stream]")
        else:
            table_at = self._ints("table_out", table_out, None)
        if lens_out is None:
            lens_out = torch.empty_like(lens)
            out_at = lens_out.data_ptr()
        else:
            out_at = self._ints("lens_out", lens_out, self.n_streams)
        if self.n_streams * self.pages_per_stream > self.n_pages:
            raise ValueError("reorder: needs pages_per_stream pages of the pool for every stream")
        launch(self.device.index, self._reorder, "talker_kv4_reorder", self._ref, at, R, lens_at, table_at, out_at)
        return self._with_table(table_out), lens_out

    def _with_table(self, page_table) -> "KV4Cache":
        """This cache under another page table of the same shape."""
        other = KV4Cache.__new__(KV4Cache)
        other.__dict__.update(self.__dict__)
        other.page_table = page_table
        other._c = _Cache.from_buffer_copy(self._c)
        other._c.page_table = page_table.data_ptr()
        other._ref = ctypes.addressof(other._c)
        return other

    def sync_status(self) -> int:
        """Wait for the device and return the status word, which is cleared (0: nothing to report)."""
        code = int(self.status.item())
        if code:
            self.status.zero_()
        return code


def _dense_heads(t):
    """t with each row's heads behind one another, itself where they are."""
    stride = t.stride()
    return t if stride[2] == 1 and (stride[1] == t.shape[2] or t.shape[1] == 1) else t.contiguous()
