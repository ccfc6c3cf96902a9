"""What the wrappers of single calls share: data types, pointers, the stream
and device of a call, and the error of a status."""
from __future__ import annotations

import contextlib

import torch
from torch.autograd import forward_ad

from . import _lib
from ._lib import CEError

DTYPES = {torch.float32: _lib.CE_F32, torch.bfloat16: _lib.CE_BF16, torch.float16: _lib.CE_F16}
_HERE = contextlib.nullcontext()


def ptr(t):
    return None if t is None else t.data_ptr()


def plain(t):
    """t's values in contiguous memory (a negation that a view defers, as that
    of z.conj().imag does, is carried out)."""
    t = t.contiguous()
    return t.resolve_neg() if t.is_neg() else t


# The current stream as an integer; the plain call builds a Stream object
# first (some microseconds, as much as the rest of a short call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream(device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def once(name, dy):
    """Refuses a backward that is itself to be differentiated, in either mode."""
    if torch.is_grad_enabled() or (
            forward_mode() and forward_ad.unpack_dual(dy).tangent is not None):
        raise RuntimeError(f"{name} is differentiable once: its backward has no graph")


def forward_mode():
    """Whether forward-mode derivatives are being taken. A tensor with a tangent
    need not require a gradient, so calls then go through their autograd
    Function, which refuses it (none has a forward-mode rule)."""
    return forward_ad._current_level >= 0


# (a CUDA tensor is at hand, so CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def on(device):
    """A context in which `device` is the current one (free where it is already)."""
    return _HERE if device.index == _current_device() else torch.cuda.device(device)


def check(rc, where):
    if rc != _lib.CE_OK:
        raise CEError(rc, where)


def require_cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
