"""One step of beam search: the selection over beams and vocabulary, and the
reordering of the beams' states.

    best = beam_search_step(logits, scores, num_candidates=2 * K, finished=done)
    beam_reorder(cache, best.beams[:, :K], inplace=True)

The definitions are those of ce_beam_select and ce_beam_reorder
(include/gbce.h). Runs in libgbce.so; there is no CPU fallback.
"""
from __future__ import annotations

from collections import namedtuple

import torch
from torch.autograd import forward_ad

from . import _lib
from ._tensors import DTYPES, check, forward_mode, on, plain, ptr, require_cuda, stream

__all__ = ["beam_search_step", "beam_reorder", "BeamCandidates"]

BeamCandidates = namedtuple("BeamCandidates", ["scores", "beams", "tokens"])


def beam_search_step(logits, scores, num_candidates=None, finished=None, pad_token=0):
    """The num_candidates (default K, at most 64) best continuations of each
    batch entry: BeamCandidates of scores (float32), beams and tokens (int64),
    each [B, num_candidates], by descending score, equal ones by the lowest
    beam, then token. logits [B, K, V] in float32, bfloat16 or float16, K at
    most 32, B and V at most 2^20; scores [B, K] float32, the beams'
    log-probabilities so far. Gradients are not tracked.

    A candidate's score is scores[b, k] + log_softmax(logits[b, k])[v]. Tokens
    whose logit is -inf or NaN are left out; a beam whose score is not finite,
    or that has no token left, offers nothing. finished [B, K] (bool): such a
    beam goes on with pad_token alone, at its own score. Where candidates run
    out, scores hold -inf, beams -1 and tokens pad_token."""
    require_cuda(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be [B, K, V]")
    if logits.dtype not in DTYPES:
        raise TypeError(f"logits dtype {logits.dtype} is not supported "
                        "(float32, bfloat16, float16)")
    B, K, V = logits.shape
    dev = logits.device
    if not isinstance(scores, torch.Tensor) or tuple(scores.shape) != (B, K) or \
            scores.device != dev or scores.dtype != torch.float32:
        raise ValueError("scores must be float32 [B, K] on the logits' device")
    if finished is not None and (finished.dtype != torch.bool or tuple(finished.shape) != (B, K) or
                                 finished.device != dev):
        raise ValueError("finished must be bool [B, K] on the logits' device")
    M = K if num_candidates is None else int(num_candidates)
    if M < 1 or K < 1 or V < 1:
        raise ValueError("num_candidates, K and V must be at least 1")
    if not 0 <= int(pad_token) < V:
        raise ValueError("pad_token must lie in [0, V)")
    logits = plain(logits)
    scores = plain(scores)
    finished = None if finished is None else finished.contiguous()
    out = BeamCandidates(torch.empty((B, M), dtype=torch.float32, device=dev),
                         torch.empty((B, M), dtype=torch.int64, device=dev),
                         torch.empty((B, M), dtype=torch.int64, device=dev))
    dt = DTYPES[logits.dtype]
    with on(dev):
        nbytes = _lib.ce_beam_workspace_bytes(dt, B, K, V, M)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
        check(_lib.ce_beam_select(ptr(logits), dt, B, K, V, ptr(scores), ptr(finished),
                                  int(pad_token), M, ptr(out.scores), ptr(out.beams),
                                  ptr(out.tokens), ptr(ws), nbytes, stream(dev)), "ce_beam_select")
    return out


def _blocks(t, skip):
    """(row stride, block stride, blocks, block elements): the dimensions of t
    behind the first `skip` as equally spaced blocks of contiguous elements."""
    inner, blocks, block_stride = 1, 1, 0
    for n, s in zip(reversed(t.shape[skip:]), reversed(t.stride()[skip:])):
        if n == 1:
            continue
        if blocks == 1 and s == inner:
            inner *= n
        elif blocks == 1:
            blocks, block_stride = n, s
        elif s == block_stride * blocks:
            blocks *= n
        else:
            raise ValueError("a state's rows must be equally spaced blocks of contiguous elements")
    # (a dimension of one, such as the beams' at K = 1, has a stride that says nothing)
    row = t.stride(0) if skip == 1 or t.shape[1] == 1 else t.stride(1)
    if skip == 2 and t.shape[0] > 1 and t.stride(0) != t.shape[1] * row:
        raise ValueError("a state's batch and beam dimensions must be one evenly spaced dimension")
    if block_stride < 0 or row < 0 or (blocks > 1 and block_stride < inner):
        raise ValueError("a state's elements must not overlap")
    return row, block_stride, blocks, inner


def beam_reorder(states, beams, inplace=False):
    """states[b, j] = states[b, beams[b, j]] for a tensor or a sequence of
    tensors of beams' states, each [B, K, ...] or [B * K, ...], of any dtype.
    beams [B, K] int64 on their device, K at most 32; a value outside [0, K) (such as the -1
    of a place without a candidate) keeps row j as it is.

    Returns new tensors, or with inplace=True changes the states and returns
    them (rows that keep their state are not touched). Strided states, such as
    cache[:, :, :length], are taken when their rows are equally spaced blocks
    of contiguous elements (ValueError otherwise). States that are changed in
    place must not overlap one another (beams may lie in one of them). The
    states' gradients are not tracked."""
    one = isinstance(states, torch.Tensor)
    states = [states] if one else list(states)
    require_cuda(beams, "beams")
    if beams.dim() != 2 or beams.dtype != torch.int64:
        raise ValueError("beams must be int64 [B, K]")
    B, K = beams.shape
    if K < 1:
        raise ValueError("beams must hold at least one beam")
    dev = beams.device
    if beams.stride(1) != 1 or beams.stride(0) < K:
        beams = beams.contiguous()
    beams_row = beams.stride(0) if B > 1 else K  # (the stride of a dimension of one says nothing)
    beams_at = beams.data_ptr()
    beams_end = beams_at + 8 * ((B - 1) * beams_row + K)
    dual, shared = inplace and forward_mode(), False
    outs, table = [], []
    for t in states:
        require_cuda(t, "a state")
        if t.device != dev:
            raise ValueError("the states must be on the beams' device")
        shape = t.shape
        skip = 2 if len(shape) >= 2 and shape[0] == B and shape[1] == K else 1
        if skip == 1 and (len(shape) < 1 or shape[0] != B * K):
            raise ValueError("a state must be [B, K, ...] or [B * K, ...]")
        if inplace and t.requires_grad:
            raise ValueError("a state that requires a gradient cannot be reordered in place")
        if dual and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError("a state with a tangent cannot be reordered in place")
        if not inplace and (t.is_conj() or t.is_neg()):
            t = t.resolve_conj().resolve_neg()  # (in place the view stays one)
        n = t.numel()
        if t.is_contiguous():
            row = inner = n // (B * K) if n else 0
            block_stride, blocks = 0, 1
        else:
            row, block_stride, blocks, inner = _blocks(t, skip)
            apart = row >= (blocks - 1) * block_stride + inner or (
                blocks > 1 and row >= inner and block_stride >= B * K * row)
            if inplace and B * K > 1 and n and not apart:
                raise ValueError("a state's rows must not overlap")
        out = t if inplace else torch.empty(shape, dtype=t.dtype, device=dev)
        outs.append(out)
        if n:
            b = t.element_size()
            to = (row * b, block_stride * b) if inplace else (blocks * inner * b, inner * b)
            src = t.data_ptr()
            table.append((src, out.data_ptr(), row * b, block_stride * b, *to, blocks, inner * b))
            if inplace and src < beams_end and beams_at < src + b * (
                    (B * K - 1) * row + (blocks - 1) * block_stride + inner):
                shared = True
    n = len(table)
    if len({at[1] for at in table}) < n:
        raise ValueError("a state is given twice")
    if shared:  # beams that lie among a state's rows would be read while these change
        beams, beams_row = beams.clone(memory_format=torch.contiguous_format), K
    table = (_lib.BeamState * n)(*table)
    with on(dev):
        check(_lib.ce_beam_reorder(table, n, ptr(beams), beams_row, B, K, stream(dev)),
              "ce_beam_reorder")
    if inplace:  # a backward that saved a state then finds that it was changed
        torch.autograd.graph.increment_version([t for t in outs if not t.is_inference()])
    return outs[0] if one else outs
