"""Verification of drafted tokens (include/talker_draft.h, talker_draft_verify)."""
from __future__ import annotations

import torch

from .kv4 import _DTYPE, contiguous_rows, launch
from .talker import load_library

_scratch = {}     # scratch bytes by (n_seq, n_draft, vocab)


def draft_verify(target_logits, tokens, uniforms, draft_logits=None, counts=None, temperatures=None):
    """Speculative decoding's decision: tokens int32 [n_seq, n_draft] drafted for each sequence are taken or refused by
    target_logits f32 or bf16 [n_seq, n_draft + 1, vocab] and the given uniforms f32 [n_seq, n_draft + 1], and the next
    token is drawn (the last uniform number of a sequence).

    draft_logits [n_seq, n_draft, vocab], of target_logits' type: what the drafts were drawn from, at the same
    temperature (None: the draft is certain of its tokens). counts int32 [n_seq]: how many drafts there are (None:
    n_draft). temperatures f32 [n_seq] (None: 1; 0 is greedy: a draft is taken if it is the target's largest logit).
    Logits lie in any strides with contiguous vocabularies. Returns tokens int32 [n_seq, n_draft + 1] (those taken, the next one, then -1), the
    number taken int32 [n_seq], and the log-probabilities of the tokens f32 [n_seq, n_draft + 1] (0 for those of -1)."""
    shape, dtype, device = target_logits.shape, _DTYPE.get(target_logits.dtype), target_logits.device
    if len(shape) != 3 or dtype is None or device.type != "cuda" or not contiguous_rows(target_logits):
        raise ValueError("draft_verify: target_logits must be an f32 or bf16 CUDA tensor [n_seq, n_draft + 1, vocab] with "
                         "contiguous vocabularies")
    n_seq, n_draft, vocab = shape[0], shape[1] - 1, shape[2]
    if not 0 <= n_draft <= 64 or vocab < 1:
        raise ValueError("draft_verify: needs at most 64 drafts and a vocabulary")
    if tokens.shape != (n_seq, n_draft) or tokens.dtype is not torch.int32 or tokens.device != device or not tokens.is_contiguous():
        raise ValueError("draft_verify: tokens must be contiguous int32 [n_seq, n_draft] on %s" % device)
    if uniforms.shape != (n_seq, n_draft + 1) or uniforms.dtype is not torch.float32 or uniforms.device != device or \
            not uniforms.is_contiguous():
        raise ValueError("draft_verify: uniforms must be contiguous f32 [n_seq, n_draft + 1] on %s" % device)
    d_at, d_seq, d_row = None, 0, 0
    if draft_logits is not None and n_draft > 0:
        if draft_logits.shape != (n_seq, n_draft, vocab) or draft_logits.dtype is not target_logits.dtype or \
                draft_logits.device != device or not contiguous_rows(draft_logits):
            raise ValueError("draft_verify: draft_logits must be [n_seq, n_draft, vocab] in target_logits' type with "
                             "contiguous vocabularies")
        d_at, (d_seq, d_row, _) = draft_logits.data_ptr(), draft_logits.stride()
    if counts is not None and (counts.shape != (n_seq,) or counts.dtype is not torch.int32 or counts.device != device or
                               not counts.is_contiguous()):
        raise ValueError("draft_verify: counts must be contiguous int32 [n_seq] on %s" % device)
    if temperatures is not None and (temperatures.shape != (n_seq,) or temperatures.dtype is not torch.float32 or
                                     temperatures.device != device or not temperatures.is_contiguous()):
        raise ValueError("draft_verify: temperatures must be contiguous f32 [n_seq] on %s" % device)
    out = torch.empty((n_seq, n_draft + 1), dtype=torch.int32, device=device)
    accepted = torch.empty((n_seq,), dtype=torch.int32, device=device)
    logprobs = torch.empty((n_seq, n_draft + 1), dtype=torch.float32, device=device)
    if n_seq == 0:
        return out, accepted, logprobs
    lib = load_library()
    need = _scratch.get((n_seq, n_draft, vocab))
    if need is None:
        if len(_scratch) >= 256:
            _scratch.clear()
        need = _scratch[(n_seq, n_draft, vocab)] = lib.talker_draft_scratch(n_seq, n_draft, vocab)
    scratch = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    t_seq, t_row, _ = target_logits.stride()
    launch(device.index, lib.talker_draft_verify, "talker_draft_verify", target_logits.data_ptr(), t_seq, t_row, d_at, d_seq, d_row,
           dtype, tokens.data_ptr(), None if counts is None else counts.data_ptr(), uniforms.data_ptr(),
           None if temperatures is None else temperatures.data_ptr(), n_seq, n_draft, vocab, out.data_ptr(),
           accepted.data_ptr(), logprobs.data_ptr(), scratch.data_ptr() if need else None, need)
    return out, accepted, logprobs
