"""The global gradient norm over many tensors, and clipping.

    norm = snack_grad_norm(grads)                       # sqrt of the sum of all squares
    norm = snack_clip_grad_norm(grads, max_norm)        # and grads *= min(1, max_norm / (norm + eps))

``grads`` is a list of CUDA tensors (float32, bfloat16, float16, mixed) or a
``SnackTensorList`` of them.  A list is checked on every call; a
``SnackTensorList`` was checked when it was made and costs a call nothing per
tensor: keep one where the gradients stay in place from step to step
(``zero_grad(set_to_none=False)``, a flat buffer, a captured graph).
"""

from __future__ import annotations

import ctypes
import math

import numpy as np
import torch

from . import _DTYPES, _abi, _check, _lib, _stream

_I64, _I32 = ctypes.c_int64, ctypes.c_int32


class SnackTensorList:
    """A list of CUDA tensors, checked once.  It holds the tensors, so their
    memory stays theirs; what they contain may change at any time."""

    def __init__(self, tensors):
        ts = list(tensors)
        for i, t in enumerate(ts):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DTYPES:
                raise TypeError(f"tensor {i} must be a CUDA float32, bfloat16 or float16 tensor")
            if not t.is_contiguous():
                raise ValueError(f"tensor {i} must be contiguous")
        self.device = ts[0].device if ts else torch.device("cuda", torch.cuda.current_device())
        if any(t.device != self.device for t in ts):
            raise ValueError("all tensors must be on one device")
        self.tensors = ts
        self.sizes = np.fromiter((t.numel() for t in ts), np.int64, len(ts))
        self._ptr = np.fromiter((t.data_ptr() for t in ts), np.uint64, len(ts))
        self._type = np.fromiter((_DTYPES[t.dtype] for t in ts), np.int32, len(ts))
        self.count = len(ts)
        self.ptr, self.size, self.type = (a.ctypes.data for a in (self._ptr, self.sizes, self._type))

    def __len__(self):
        return self.count


def snack_tensor_list(tensors) -> SnackTensorList:
    """Check a list of tensors once, for many calls."""
    return tensors if isinstance(tensors, SnackTensorList) else SnackTensorList(tensors)


def _prepare(grads, norm_type, norm):
    lst = snack_tensor_list(grads)
    if norm_type == 2.0:
        kind = 0
    elif norm_type == math.inf:
        kind = 1
    else:
        raise ValueError("norm_type must be 2.0 or inf")
    if lst.device.index != torch.cuda.current_device():
        raise ValueError(f"{lst.device} is not the current CUDA device")
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=lst.device)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != lst.device:
        raise ValueError("norm must be one float32 on the gradients' device")
    ws = torch.empty(_lib.snack_grad_norm_workspace(lst.count), dtype=torch.uint8,
                     device=lst.device)
    return lst, kind, norm, ws


def snack_grad_norm(grads, norm_type: float = 2.0, norm: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The norm of all tensors together (2.0 or inf), as one float32 on the device."""
    lst, kind, norm, ws = _prepare(grads, norm_type, norm)
    s = _stream(stream, lst.device)
    _record(ws, stream)
    _check(_lib.snack_grad_norm(lst.count, lst.ptr, lst.size, lst.type, kind, norm.data_ptr(),
                                ws.data_ptr(), s))
    return norm


def snack_clip_grad_norm(grads, max_norm: float, norm_type: float = 2.0, out=None,
                         eps: float = 1e-6, norm: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Scale the gradients by min(1, max_norm / (norm + eps)) and return their
    norm before that, as one float32 on the device.  In place, or into ``out``
    (a list or SnackTensorList of the same sizes; its types may differ, e.g.
    float32 buffers of an optimizer for bfloat16 gradients).  A NaN norm makes
    every result NaN; an infinite one zeros what is finite."""
    lst, kind, norm, ws = _prepare(grads, norm_type, norm)
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError("max_norm must be >= 0")
    outs = types = None
    if out is not None:
        o = snack_tensor_list(out)
        if o.count != lst.count or not np.array_equal(o.sizes, lst.sizes):
            raise ValueError("out must hold as many elements as grads, tensor by tensor")
        if o.count and o.device != lst.device:
            raise ValueError("all tensors must be on one device")
        outs, types = o.ptr, o.type
    s = _stream(stream, lst.device)
    _record(ws, stream)
    _check(_lib.snack_clip_grad_norm(lst.count, lst.ptr, outs, lst.size, lst.type, types, kind,
                                     max_norm, eps, norm.data_ptr(), ws.data_ptr(), s))
    return norm


def _record(ws: torch.Tensor, stream) -> None:
    """Scratch used on a stream that is not the current one stays reserved until that work is done."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=ws.device)
        ws.record_stream(stream)
