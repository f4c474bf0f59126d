"""Dropout whose mask is a function of a seed and is never stored.

    y = residual + M * x        (without a residual: M * x)

M is 0 for a share p of the elements and 1 / (1 - p) for the others; p counts
in steps of 2^-16.  The gradient of x is M times that of y, with the mask
made again from the same seed.  ``seed`` is a number, or one int64 on the
device that is read when the kernel runs: a captured graph draws new masks
where it also changes that tensor.  Tensors of unlike content need unlike
seeds: element e of every tensor takes the same draw of a seed.
"""

from __future__ import annotations

import torch

from . import _dense, _raw_stream
from ._autograd import first_derivative


def snack_dropout_forward(x: torch.Tensor, p: float, seed, residual: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """y of the residual's type (x's without one).  x and residual contiguous, of one shape."""
    return _dense.dropout(x, residual, None, p, seed, _raw_stream(stream))


def snack_dropout_backward(dy: torch.Tensor, p: float, seed, dtype=None,
                           stream=None) -> torch.Tensor:
    """The gradient of x (of type ``dtype``, by default dy's) for the same p and seed."""
    return _dense.dropout(dy, None, dtype, p, seed, _raw_stream(stream))


class _DropoutFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed):
        y = snack_dropout_forward(x.contiguous(), p, seed,
                                  None if residual is None else residual.contiguous())
        ctx.p, ctx.dtype = p, x.dtype
        ctx.seed = None if isinstance(seed, torch.Tensor) else seed
        ctx.save_for_backward(*([seed] if ctx.seed is None else []))
        return y

    @staticmethod
    @first_derivative
    def backward(ctx, dy):
        seed = ctx.saved_tensors[0] if ctx.seed is None else ctx.seed
        dx = snack_dropout_backward(dy.contiguous(), ctx.p, seed, ctx.dtype) \
            if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None


def snack_dropout(x: torch.Tensor, p: float, seed, residual: torch.Tensor | None = None) -> torch.Tensor:
    """residual + M * x (or M * x) with gradients."""
    return _DropoutFunction.apply(x, residual, p, seed)
