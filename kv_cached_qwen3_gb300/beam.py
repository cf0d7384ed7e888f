"""Beam selection (include/talker_kv4.h, talker_beam_select)."""
from __future__ import annotations

import torch

from .kv4 import _DTYPE, launch
from .talker import load_library

_scratch = {}     # scratch bytes by the logits' shape


def beam_select(logits, scores, ended=None, eos_id: int = -1):
    """The best `width` continuations of each sequence: logits [n_seq, width, vocab] f32 or bf16 (rows at one
    stride), scores [n_seq, width] f32, ended [n_seq, width] int32 or None. A continuation's score is the beam's plus
    the token's log-probability; an ended beam has only eos_id, at its unchanged score. Returns tokens, parents
    (int32 row numbers seq * width + beam), scores and ended flags, each [n_seq, width], best first."""
    shape, stride, dtype, device = logits.shape, logits.stride(), _DTYPE.get(logits.dtype), logits.device
    if len(shape) != 3 or dtype is None or device.type != "cuda":
        raise ValueError("beam_select: logits must be an f32 or bf16 CUDA tensor [n_seq, width, vocab]")
    n_seq, width, vocab = shape
    if not 1 <= width <= 32 or vocab < width:
        raise ValueError("beam_select: width must be 1 to 32 and at most vocab")
    if eos_id >= vocab or (ended is not None and eos_id < 0):
        raise ValueError("beam_select: eos_id must be a token of the vocabulary")
    if scores.shape != (n_seq, width) or scores.dtype is not torch.float32 or scores.device != device or \
            not scores.is_contiguous():
        raise ValueError("beam_select: scores must be contiguous f32 [n_seq, width] on %s" % device)
    if ended is not None and (ended.shape != (n_seq, width) or ended.dtype is not torch.int32 or ended.device != device
                              or not ended.is_contiguous()):
        raise ValueError("beam_select: ended must be contiguous int32 [n_seq, width] on %s" % device)
    row = stride[1] if width > 1 else stride[0]
    if stride[2] != 1 or row < vocab or (n_seq > 1 and stride[0] != width * row):
        logits, row = logits.contiguous(), vocab
    out = (n_seq, width)
    tokens, parents, done = (torch.empty(out, dtype=torch.int32, device=device) for _ in range(3))
    best = torch.empty(out, dtype=torch.float32, device=device)
    if n_seq == 0:
        return tokens, parents, best, done
    lib = load_library()
    need = _scratch.get(shape)
    if need is None:
        if len(_scratch) >= 256:
            _scratch.clear()
        need = _scratch[shape] = lib.talker_beam_scratch(n_seq, width, vocab)
    scratch = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    launch(device.index, lib.talker_beam_select, "talker_beam_select", logits.data_ptr(), row, dtype, scores.data_ptr(),
           None if ended is None else ended.data_ptr(), n_seq, width, vocab, eos_id, tokens.data_ptr(),
           parents.data_ptr(), best.data_ptr(), done.data_ptr(), scratch.data_ptr() if need else None, need)
    return tokens, parents, best, done
