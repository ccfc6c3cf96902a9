"""Dropout from a counter-based generator, with the residual sum fused in.

    y = dropout(x, p, seed, offset=0, residual=None)

y = residual + keep * x / (1 - p). Whether element i is kept is a function of
(p, seed, offset, i) alone (Philox 4x32-10; see ce_dropout in
include/gbce.h), so the backward forms the words again and no mask is
stored. Runs in libgbce.so; there is no CPU fallback.
"""
from __future__ import annotations

import torch

from . import _lib
from ._tensors import DTYPES, check, forward_mode, on, once, plain, ptr, require_cuda, stream

__all__ = ["dropout", "DropoutFunction"]

_U64 = (1 << 64) - 1


def check_rng(p, seed, offset, device):
    """(p, seed, offset, state): the arguments of dropout as the library takes
    them. A seed tensor is passed on where words are drawn from it (p not 0 or 1)."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError("the dropout probability must lie in [0, 1]")
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 2 or seed.device != device:
            raise ValueError("a seed tensor holds int64 (seed, offset) on the input's device")
        return p, 0, int(offset) & _U64, seed.contiguous() if 0.0 < p < 1.0 else None
    if seed is None:
        if p not in (0.0, 1.0):
            raise ValueError("dropout needs a seed")
        seed = 0
    return p, int(seed) & _U64, int(offset) & _U64, None


def _call(x, residual, p, seed, offset, state, used):
    y = torch.empty_like(x)
    dev = x.device
    with on(dev):
        check(_lib.ce_dropout(ptr(x), ptr(residual), ptr(y), DTYPES[x.dtype], x.numel(), p, seed,
                              offset, ptr(state), ptr(used), stream(dev)), "ce_dropout")
    return y


class DropoutFunction(torch.autograd.Function):
    """Autograd wrapper of ce_dropout: the backward is the same call on grad_output."""

    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, state):
        used = None
        if state is not None and ctx.needs_input_grad[0]:
            # the caller may change the state before the backward runs
            used = torch.empty(2, dtype=torch.int64, device=x.device)
            ctx.save_for_backward(used)
        ctx.rng = (p, seed, offset)
        return _call(x, residual, p, seed, offset, state, used)

    @staticmethod
    def backward(ctx, dy):
        once("dropout", dy)
        dx = None
        if ctx.needs_input_grad[0]:
            p, seed, offset = ctx.rng
            used = ctx.saved_tensors[0] if ctx.saved_tensors else None
            if used is not None:
                offset = 0  # in `used` already
            dx = _call(plain(dy), None, p, seed, offset, used, None)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None, None


def dropout(x, p, seed, offset=0, residual=None):
    """residual + x with each element dropped with probability p, the others
    scaled by 1 / (1 - p). x (any shape) in float32, bfloat16 or float16 on
    CUDA; residual None or like x. Differentiable once, in reverse mode.

    seed: an int, or an int64 CUDA tensor (seed, offset) that the kernel reads
    when it runs (its offset is added to `offset`): a captured graph then draws
    other elements on each replay when the program updates the tensor between
    them. Draw (seed, offset) pairs apart for calls that must be independent:
    calls with the same pair drop the same elements."""
    require_cuda(x, "x")
    if x.dtype not in DTYPES:
        raise TypeError(f"x dtype {x.dtype} is not supported (float32, bfloat16, float16)")
    if residual is not None:
        require_cuda(residual, "residual")
        if residual.shape != x.shape or residual.dtype != x.dtype or residual.device != x.device:
            raise ValueError("residual must have the shape, dtype and device of x")
        residual = plain(residual)
    p, seed, offset, state = check_rng(p, seed, offset, x.device)
    x = plain(x)
    if not (forward_mode() or (torch.is_grad_enabled() and (
            x.requires_grad or (residual is not None and residual.requires_grad)))):
        return _call(x, residual, p, seed, offset, state, None)
    return DropoutFunction.apply(x, residual, p, seed, offset, state)
