"""What the autograd functions of the dense operators share."""

from __future__ import annotations

import functools

import torch


class _Once(torch.autograd.Function):
    """A gradient that must not be differentiated again."""

    @staticmethod
    def forward(ctx, g):
        return g.view_as(g)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("second derivatives of this operator are not implemented")


def first_derivative(backward):
    """A Function's backward whose results come from kernels that autograd
    does not see.  Under create_graph=True they would count as constants, and
    second derivatives would lack their terms in silence: here differentiating
    them raises, whatever the incoming gradients."""

    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        return tuple(None if g is None else _Once.apply(g.detach().requires_grad_()) for g in out)

    return wrapped
