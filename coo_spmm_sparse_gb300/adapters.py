"""Low-rank adapters of many requests at once beside one projection.

Request i owns the tokens offsets[i] .. offsets[i+1]-1 of X and names adapter
n = adapter[i] (-1: none).  For each of its tokens

    H[t] = A[n] X[t],    Y[t] += scale[n] * B[n] H[t]

Y arrives with the shared projection's output (``snack_forward``) and leaves
with the adapters' part added.  ``SnackAdapters`` keeps the weights of the
adapters of one projection and carries the gradients.
"""

from __future__ import annotations

import math

import torch

from . import _dense, _raw_stream
from ._autograd import first_derivative


def snack_adapter_forward(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                          offsets: torch.Tensor, adapter: torch.Tensor, scale, Y: torch.Tensor,
                          H: torch.Tensor | None = None, stream=None):
    """Add the adapters' part to Y in place; returns (Y, H) with H [tokens][rank] float32.

    X [..., in] and Y [..., out] may have strided rows; A [adapters][rank][in],
    B [adapters][out][rank]; offsets [requests + 1] and adapter [requests] int32
    on the device (not read by the host); scale a number or float32 [adapters]."""
    return _dense.adapter_forward(X, A, B, offsets, adapter, scale, Y, H, _raw_stream(stream))


def snack_adapter_backward(X: torch.Tensor, dY: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                           offsets: torch.Tensor, adapter: torch.Tensor, scale, H: torch.Tensor,
                           dX: torch.Tensor | None = None, need_dx: bool = True,
                           need_dw: bool = True, stream=None):
    """(dX, dA, dB) of the adapters' part of Y.  dX is added to in place where
    it is given (the projection's own input gradient), else started from
    zeros; dA and dB have the shapes of A and B."""
    return _dense.adapter_backward(X, dY, A, B, offsets, adapter, scale, H, dX, need_dx, need_dw,
                                   _raw_stream(stream))


class _AdapterFunction(torch.autograd.Function):
    """Y of the projection with the adapters' part added in place."""

    @staticmethod
    def forward(ctx, X, Y, A, B, offsets, adapter, scale):
        if ctx.needs_input_grad[6]:
            raise ValueError("scale has no gradient here: detach it, or scale B")
        _, H = snack_adapter_forward(X, A, B, offsets, adapter, scale, Y)
        ctx.mark_dirty(Y)
        ctx.scale = scale
        ctx.save_for_backward(X, A, B, offsets, adapter, H)
        return Y

    @staticmethod
    @first_derivative
    def backward(ctx, dY):
        X, A, B, offsets, adapter, H = ctx.saved_tensors
        need = ctx.needs_input_grad
        if need[0] or need[2] or need[3]:
            dX, dA, dB = snack_adapter_backward(X, dY.contiguous(), A, B, offsets, adapter,
                                                ctx.scale, H, need_dx=need[0],
                                                need_dw=need[2] or need[3])
        else:
            dX = dA = dB = None
        return dX, dY, dA if need[2] else None, dB if need[3] else None, None, None, None


class SnackAdapters(torch.nn.Module):
    """The adapters of one projection: A [adapters][rank][in] drawn N(0, 1/in),
    B [adapters][out][rank] zero, so that a new adapter changes nothing.

    ``forward(x, y, offsets, adapter)`` adds their part to the projection's
    output y (in place) and returns it.  ``scale`` is alpha / rank; it may be
    set to another number or to float32 [adapters] that wants no gradient."""

    def __init__(self, adapters: int, in_features: int, out_features: int, rank: int,
                 alpha: float | None = None, seed: int = 0, dtype=torch.float32, device=None):
        super().__init__()
        dev = device or torch.device("cuda", torch.cuda.current_device())
        g = torch.Generator(device="cpu").manual_seed(seed)
        a = torch.randn(adapters, rank, in_features, generator=g) / math.sqrt(in_features)
        self.A = torch.nn.Parameter(a.to(dev, dtype))
        self.B = torch.nn.Parameter(torch.zeros(adapters, out_features, rank, device=dev,
                                                dtype=dtype))
        self.scale = 1.0 if alpha is None else alpha / rank

    def forward(self, x: torch.Tensor, y: torch.Tensor, offsets: torch.Tensor,
                adapter: torch.Tensor) -> torch.Tensor:
        return _AdapterFunction.apply(x, y, self.A, self.B, offsets, adapter, self.scale)
