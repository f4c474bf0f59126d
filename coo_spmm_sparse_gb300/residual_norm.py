"""The norms before and after a block, with its gate and residual scales.

    u = P(y) or y
    r = residual_scale * x + branch_scale * gate * u
    h = N(r)

x is the residual stream, y a block's output, r the next residual and h what
the next block reads; P (``post_norm``) and N (``next_norm``) are layer norms
("layer") or root-mean-square norms ("rms") over the last dimension.  With
y = None it is a plain norm of x.
"""

from __future__ import annotations

import torch

from . import _dense, _raw_stream
from ._autograd import first_derivative

_KINDS = {"layer": 0, "rms": 1}


def _kind(kind):
    if kind not in _KINDS:
        raise ValueError("kind must be 'layer' or 'rms'")
    return _KINDS[kind]


def snack_residual_norm_forward(x: torch.Tensor, y: torch.Tensor | None = None, *,
                                kind: str = "layer", post_norm: bool = False,
                                post_weight=None, post_bias=None, gate=None,
                                residual_scale: float = 1.0, branch_scale: float = 1.0,
                                next_norm: bool = True, next_weight=None, next_bias=None,
                                eps: float = 1e-5, branch_dtype=None, stream=None):
    """(r, h, stats).  r has x's type, h y's (``branch_dtype`` where y is None);
    r is x itself where nothing is added to it, h is None without ``next_norm``.
    gate: [d], [..., 1] (per token), [sequences, 1, d] or x's shape, of y's
    type.  stats [rows][4] float32 is what the backward call reads."""
    return _dense.norm_forward(x, y, gate, post_weight, post_bias, next_weight, next_bias,
                               _kind(kind), post_norm, next_norm, residual_scale, branch_scale,
                               eps, branch_dtype, _raw_stream(stream))


def snack_residual_norm_backward(dr, dh, x: torch.Tensor, y: torch.Tensor | None,
                                 stats: torch.Tensor, *, kind: str = "layer",
                                 post_norm: bool = False, post_weight=None, post_bias=None,
                                 gate=None, residual_scale: float = 1.0,
                                 branch_scale: float = 1.0, next_norm: bool = True,
                                 next_weight=None, next_bias=None, eps: float = 1e-5,
                                 branch_dtype=None, stream=None) -> dict:
    """Gradients of (r, h) -> dict with "dx", "dy", "dgate", "dpost_weight",
    "dpost_bias", "dnext_weight", "dnext_bias" for the inputs that are there.
    dr or dh may be None (zero).  The options are those of the forward call
    that returned ``stats``."""
    return _dense.norm_backward(dr, dh, x, y, stats, gate, post_weight, post_bias, next_weight,
                                next_bias, _kind(kind), post_norm, next_norm, residual_scale,
                                branch_scale, eps, branch_dtype, _raw_stream(stream))


class _ResidualNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, gate, post_weight, post_bias, next_weight, next_bias, opts):
        r, h, stats = snack_residual_norm_forward(
            x, y, gate=gate, post_weight=post_weight, post_bias=post_bias,
            next_weight=next_weight, next_bias=next_bias, **opts)
        ctx.opts = opts
        ctx.save_for_backward(x, y, gate, post_weight, post_bias, next_weight, next_bias, stats)
        ctx.set_materialize_grads(False)
        return (r.view_as(r) if r is x else r), h

    @staticmethod
    @first_derivative
    def backward(ctx, dr, dh):
        x, y, gate, pw, pb, nw, nb, stats = ctx.saved_tensors
        if dr is None and dh is None:
            return (None,) * 8
        g = snack_residual_norm_backward(
            None if dr is None else dr.contiguous(), None if dh is None else dh.contiguous(), x, y,
            stats, gate=gate, post_weight=pw, post_bias=pb, next_weight=nw, next_bias=nb,
            **ctx.opts)
        keys = ("dx", "dy", "dgate", "dpost_weight", "dpost_bias", "dnext_weight", "dnext_bias")
        return tuple(g.get(k) if need else None
                     for k, need in zip(keys, ctx.needs_input_grad)) + (None,)


def snack_residual_norm(x, y=None, *, gate=None, post_weight=None, post_bias=None,
                        next_weight=None, next_bias=None, **opts):
    """(r, h) with gradients; the options of snack_residual_norm_forward."""
    return _ResidualNormFunction.apply(x, y, gate, post_weight, post_bias, next_weight, next_bias,
                                       opts)


class SnackResidualNorm(torch.nn.Module):
    """``r, h = norm(x, y)``: the add, gate and norms between two blocks.

    ``post``: normalise the block's output before it is added; ``gate``:
    "channel" learns one factor per channel (started at ``gate_init``), a
    tensor passed to forward is any other gate.  ``next``: whether h is
    wanted.  Layer norms have biases, rms norms have none."""

    def __init__(self, width: int, kind: str = "layer", post: bool = False, next: bool = True,
                 gate: str | None = None, gate_init: float = 1.0, residual_scale: float = 1.0,
                 branch_scale: float = 1.0, eps: float = 1e-5, dtype=torch.float32, device=None):
        super().__init__()
        dev = device or torch.device("cuda", torch.cuda.current_device())

        def param(on, value):
            return torch.nn.Parameter(torch.full((width,), value, device=dev, dtype=dtype)) \
                if on else None

        layer = kind == "layer"
        self.post_weight, self.post_bias = param(post, 1.0), param(post and layer, 0.0)
        self.next_weight, self.next_bias = param(next, 1.0), param(next and layer, 0.0)
        if gate not in (None, "channel"):
            raise ValueError("gate must be None or 'channel'")
        self.gate = param(gate == "channel", gate_init)
        self.opts = dict(kind=kind, post_norm=post, next_norm=next, eps=eps,
                         residual_scale=residual_scale, branch_scale=branch_scale)

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, gate=None):
        if gate is None and y is not None and self.gate is not None:
            gate = self.gate.to(y.dtype)
        if y is None and self.opts["post_norm"]:
            raise ValueError("a norm after the block needs the block's output")
        return snack_residual_norm(x, y, gate=gate, post_weight=self.post_weight,
                                   post_bias=self.post_bias, next_weight=self.next_weight,
                                   next_bias=self.next_bias, **self.opts)
