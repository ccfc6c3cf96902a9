"""The gated feed-forward block on the tensor cores.

    y = gated_feed_forward(x, gate_weight, up_weight, down_weight,
                           activation="silu", dropout_p=0.0, seed=None,
                           residual=None)

y = residual + dropout(h @ down_weight^T) with h = act(x @ gate_weight^T) *
(x @ up_weight^T): both projections, the activation and the product in one
kernel, dropout and the residual sum in the second's epilogue, and the whole
backward pass (ce_ffn_fwd and ce_ffn_bwd in include/gbce.h). Runs in
libgbce.so; there is no CPU fallback.
"""
from __future__ import annotations

import torch

from . import _lib
from ._tensors import DTYPES, check, forward_mode, on, once, plain, ptr, require_cuda, stream
from .philox_dropout import check_rng

__all__ = ["gated_feed_forward", "GatedFeedForward", "GatedFeedForwardFunction"]

_ACTIVATIONS = {"silu": _lib.CE_ACT_SILU, "gelu": _lib.CE_ACT_GELU,
                "gelu_tanh": _lib.CE_ACT_GELU_TANH}


def _forward(x, w_gate, w_up, w_down, residual, act, p, seed, offset, state, grad):
    """(y, h, sa): h [rows, I] in rows of whole 16-byte vectors and, with grad,
    u act'(g) and act(g) in float32 [2, rows, I] likewise, for the backward."""
    rows, H = x.shape
    O, I = w_down.shape
    dev, dt = x.device, x.dtype
    y = torch.empty((rows, O), dtype=dt, device=dev)
    I8 = (I + 7) // 8 * 8
    h = torch.empty((rows, I8), dtype=dt, device=dev)
    sa = torch.empty((2, rows, I8), dtype=torch.float32, device=dev) if grad else None
    s = sa.data_ptr() if grad else None
    a = s + rows * I8 * 4 if grad else None
    with on(dev):
        nbytes = _lib.ce_ffn_fwd_workspace_bytes(rows, H, I, O)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        check(_lib.ce_ffn_fwd(ptr(x), ptr(w_gate), ptr(w_up), ptr(w_down), ptr(residual),
                              DTYPES[dt], rows, H, I, O, act, p, seed, offset, ptr(state), ptr(y),
                              ptr(h), s, a, ptr(ws), nbytes, stream(dev)), "ce_ffn_fwd")
    return y, h, sa


class GatedFeedForwardFunction(torch.autograd.Function):
    """Autograd wrapper of ce_ffn_fwd and ce_ffn_bwd on [rows, H] inputs. The
    forward keeps x and, [rows, I] each, h and in float32 u act'(g) and act(g)."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, residual, act, p, seed, offset, state):
        grad = any(ctx.needs_input_grad[:4])
        if grad and state is not None:
            state = state.clone()  # the caller may change it before the backward runs
        y, h, sa = _forward(x, w_gate, w_up, w_down, residual, act, p, seed, offset, state, grad)
        if grad:
            ctx.save_for_backward(x, w_gate, w_up, w_down, h, sa, state)
        ctx.args = (act, p, seed, offset)
        return y

    @staticmethod
    def backward(ctx, dy):
        once("gated_feed_forward", dy)
        need = ctx.needs_input_grad
        dx = dwg = dwu = dwd = None
        if any(need[:4]):
            x, w_gate, w_up, w_down, h, sa, state = ctx.saved_tensors
            act, p, seed, offset = ctx.args
            rows, H = x.shape
            O, I = w_down.shape
            dev, dt = x.device, x.dtype
            g = aligned(dy)
            dx = torch.empty_like(x) if need[0] else None
            if need[1] or need[2]:
                dwg, dwu = torch.empty_like(w_gate), torch.empty_like(w_up)
            dwd = torch.empty_like(w_down) if need[3] else None
            nbytes = _lib.ce_ffn_bwd_workspace_bytes(rows, H, I, O, p)
            s = sa.data_ptr()
            with on(dev):
                ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
                check(_lib.ce_ffn_bwd(ptr(g), ptr(x), ptr(w_gate), ptr(w_up), ptr(w_down), ptr(h),
                                      s, s + sa.stride(0) * 4, DTYPES[dt], rows, H, I, O, act, p,
                                      seed, offset, ptr(state), ptr(dx), ptr(dwg), ptr(dwu),
                                      ptr(dwd), ptr(ws), nbytes, stream(dev)), "ce_ffn_bwd")
        return (dx, dwg if need[1] else None, dwu if need[2] else None, dwd,
                dy if need[4] else None, None, None, None, None, None)


def aligned(t):
    """t as a contiguous tensor whose base the kernels take: 16-byte aligned
    where its rows are whole 16-byte vectors."""
    t = t.contiguous()
    if t.is_neg():
        t = t.resolve_neg()
    return t.clone() if t.data_ptr() % 16 and t.shape[-1] % 8 == 0 else t


def _refuse(*tensors):
    for t in tensors:
        if t is not None:
            require_cuda(t, "every tensor of the block")
    if any(t is not None and t.device != tensors[0].device for t in tensors):
        raise ValueError("the tensors must be on one device")
    raise TypeError("the block takes bfloat16 or float16, the same for every tensor")


def gated_feed_forward(x, gate_weight, up_weight, down_weight, activation="silu", dropout_p=0.0,
                       seed=None, offset=0, residual=None):
    """residual + dropout((act(x @ gate_weight^T) * (x @ up_weight^T)) @ down_weight^T).

    x [..., H], gate_weight and up_weight [I, H], down_weight [O, I], residual
    None or [..., O], all bfloat16 or float16 on one CUDA device; activation
    "silu", "gelu" or "gelu_tanh". dropout_p, seed and offset as for dropout()
    over the [..., O] elements. Differentiable (once, in reverse mode) in x, the
    weights and residual; for that the forward keeps x and 10 bytes for each of
    the [..., I] elements. act(g) u is rounded to the tensors' type: in float16
    it is infinite above 65504, and so is what the output gets from it.

    H, I and O that are not multiples of 8 cost a packed copy of what they
    concern (x and the projections for H, down_weight for I) on each call."""
    dt, dev = x.dtype, x.device
    if not x.is_cuda or (dt != torch.bfloat16 and dt != torch.float16) or \
            gate_weight.dtype != dt or up_weight.dtype != dt or down_weight.dtype != dt or \
            gate_weight.device != dev or up_weight.device != dev or down_weight.device != dev or \
            (residual is not None and (residual.dtype != dt or residual.device != dev)):
        _refuse(x, gate_weight, up_weight, down_weight, residual)
    if gate_weight.dim() != 2 or down_weight.dim() != 2 or gate_weight.shape != up_weight.shape:
        raise ValueError("gate_weight and up_weight must be [I, H], down_weight [O, I]")
    I, H = gate_weight.shape
    O = down_weight.shape[0]
    if x.dim() < 1 or x.shape[-1] != H or down_weight.shape[1] != I or min(H, I, O) < 1:
        raise ValueError("x must be [..., H], down_weight [O, I]")
    flat = x.dim() == 2
    shape = (*x.shape[:-1], O)
    if residual is not None and residual.shape != shape:
        raise ValueError("residual must have the shape of the output")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}")
    act = _ACTIVATIONS[activation]
    p, seed, offset, state = check_rng(dropout_p, seed, offset, dev)
    if not flat:
        x = x.reshape(-1, H)
        residual = None if residual is None else residual.reshape(-1, O)
    args = (aligned(x), aligned(gate_weight), aligned(up_weight), aligned(down_weight),
            None if residual is None else plain(residual), act, p, seed, offset, state)
    if forward_mode() or (torch.is_grad_enabled() and (
            x.requires_grad or gate_weight.requires_grad or up_weight.requires_grad or
            down_weight.requires_grad or (residual is not None and residual.requires_grad))):
        y = GatedFeedForwardFunction.apply(*args)
    else:
        y = _forward(*args, False)[0]
    return y if flat else y.reshape(shape)


class GatedFeedForward(torch.nn.Module):
    """Module form of gated_feed_forward, with its three weights. Its dropout
    (in training mode) takes the seed of each call."""

    def __init__(self, hidden_size, intermediate_size, activation="silu", dropout_p=0.0,
                 device=None, dtype=torch.bfloat16):
        super().__init__()
        f = dict(device=device, dtype=dtype)
        self.gate = torch.nn.Parameter(torch.empty(intermediate_size, hidden_size, **f))
        self.up = torch.nn.Parameter(torch.empty(intermediate_size, hidden_size, **f))
        self.down = torch.nn.Parameter(torch.empty(hidden_size, intermediate_size, **f))
        self.activation = activation
        self.dropout_p = dropout_p
        self.reset_parameters()

    def reset_parameters(self):
        for w in (self.gate, self.up, self.down):
            torch.nn.init.normal_(w, std=w.shape[1] ** -0.5)

    def forward(self, x, residual=None, seed=None, offset=0):
        p = self.dropout_p if self.training else 0.0
        return gated_feed_forward(x, self.gate, self.up, self.down, self.activation, p, seed,
                                  offset, residual)
