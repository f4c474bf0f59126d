"""The global gradient norm over many tensors, and clipping.

    norm = snack_grad_norm(grads)                       # sqrt of the sum of all squares
    norm = snack_clip_grad_norm(grads, max_norm)        # and grads *= min(1, max_norm / (norm + eps))

``grads`` is a list of contiguous CUDA tensors (float32, bfloat16, float16,
mixed) or a ``SnackTensorList`` of them.  A list is checked on every call; a
``SnackTensorList`` was checked when it was made, and a call looks only at
whether its tensors are where they were: keep one where the gradients stay in
place from step to step (``zero_grad(set_to_none=False)``, a flat buffer).
A captured graph reads and writes the memory that the tensors had when it was
captured.
"""

from __future__ import annotations

import torch

from . import _dense, _raw_stream


class SnackTensorList:
    """A list of CUDA tensors, checked once.  It holds the tensors; what they
    contain may change at any time, and a tensor that was given other memory,
    another type or size is checked again by the next call.  A call that writes
    them does not move their autograd versions, as one on a list does: keep no
    list of tensors that a graph has saved."""

    __slots__ = ("tensors", "handle")

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        self.handle = _dense.tensor_list(self.tensors)

    def __len__(self):
        return len(self.tensors)


def snack_tensor_list(tensors) -> SnackTensorList:
    """Check a list of tensors once, for many calls."""
    return tensors if isinstance(tensors, SnackTensorList) else SnackTensorList(tensors)


def _handle(tensors):
    return tensors.handle if isinstance(tensors, SnackTensorList) else tensors


def snack_grad_norm(grads, norm_type: float = 2.0, norm: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The norm of all tensors together (2.0 or inf), as one float32 on the device."""
    return _dense.grad_norm(_handle(grads), norm_type, norm, _raw_stream(stream))


def snack_clip_grad_norm(grads, max_norm: float, norm_type: float = 2.0, out=None,
                         eps: float = 1e-6, norm: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Scale the gradients by min(1, max_norm / (norm + eps)) and return their
    norm before that, as one float32 on the device.  In place, or into ``out``
    (a list or SnackTensorList of the same sizes; its types may differ, e.g.
    float32 buffers of an optimizer for bfloat16 gradients).  ``out`` must not
    overlap the gradients otherwise; this is not checked.  A NaN gradient makes
    every result NaN; an infinite one zeros what is finite."""
    return _dense.clip_grad_norm(_handle(grads), max_norm, norm_type,
                                 None if out is None else _handle(out), eps, norm,
                                 _raw_stream(stream))
