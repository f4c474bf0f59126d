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

import ctypes

import torch

from . import _abi, _addr, _check, _dense_type, _lib, _rows, _same_device, _stream
from .grad_clip import _record

_KINDS = {"layer": 0, "rms": 1}
_NONE, _CHANNEL, _TOKEN, _SEQUENCE, _FULL = range(5)


def _gate_kind(gate, x):
    """(gate kind, rows that share a gate row, row stride)."""
    d = x.shape[-1]
    if tuple(gate.shape) == (d,) and x.dim() >= 1:
        if gate.stride(0) != 1 and d > 1:
            raise ValueError("gate must be contiguous")
        return _CHANNEL, 0, d
    if tuple(gate.shape) == tuple(x.shape):
        return _FULL, 0, _rows(gate, "gate")[1]
    if not gate.is_contiguous():
        raise ValueError("gate must be contiguous")
    if tuple(gate.shape) == tuple(x.shape[:-1]) + (1,):
        return _TOKEN, 0, 1
    if x.dim() >= 3 and tuple(gate.shape) == tuple(x.shape[:-2]) + (1, d):
        return _SEQUENCE, x.shape[-2], d
    raise ValueError(f"gate of shape {tuple(gate.shape)} does not fit x {tuple(x.shape)}: it is "
                     "[d], [..., 1], [sequences, 1, d] or x's shape")


def _args(x, y, kind, post_norm, post_weight, post_bias, gate, residual_scale, branch_scale,
          next_norm, next_weight, next_bias, eps, branch_dtype):
    if kind not in _KINDS:
        raise ValueError("kind must be 'layer' or 'rms'")
    st = _dense_type(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have a last dimension of at least 1")
    if y is not None:
        if _dense_type(y, "y") is not None and y.shape != x.shape:
            raise ValueError(f"y {tuple(y.shape)} must have x's shape {tuple(x.shape)}")
        branch_dtype = y.dtype
    elif post_norm or gate is not None:
        raise ValueError("post_norm and gate need y")
    elif branch_dtype is None:
        branch_dtype = x.dtype
    bt = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[branch_dtype]
    if st != bt and st != 0:
        raise TypeError("x must be float32 or have the branch's type")
    d = x.shape[-1]
    pt = None
    for t, name, used in ((post_weight, "post_weight", post_norm),
                          (post_bias, "post_bias", post_norm),
                          (next_weight, "next_weight", next_norm),
                          (next_bias, "next_bias", next_norm)):
        if t is None:
            continue
        if not used:
            raise ValueError(f"{name} without its norm")
        k = _dense_type(t, name)
        if k not in (0, bt):
            raise TypeError(f"{name} must be float32 or have the branch's type")
        if pt is not None and k != pt:
            raise TypeError("weights and biases must have one type")
        if t.numel() != d or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous vector of {d}")
        pt = k
    gk, group, gs = _NONE, 0, 0
    if gate is not None:
        if gate.dtype != branch_dtype or not gate.is_cuda:
            raise TypeError("gate must have y's type")
        gk, group, gs = _gate_kind(gate, x)
    dev = _same_device(x, y, gate, post_weight, post_bias, next_weight, next_bias)
    rows, xs = _rows(x, "x")
    ys = _rows(y, "y")[1] if y is not None else 0
    a = _abi.NormArgs(rows, d, group, _KINDS[kind], int(post_norm), int(next_norm), gk, st, bt,
                      0 if pt is None else pt, 0, residual_scale, branch_scale, eps, 0.0,
                      _addr(x), _addr(y), _addr(gate), xs, ys, gs, _addr(post_weight),
                      _addr(post_bias), _addr(next_weight), _addr(next_bias), None)
    return a, dev, branch_dtype


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
    a, dev, bdt = _args(x, y, kind, post_norm, post_weight, post_bias, gate, residual_scale,
                        branch_scale, next_norm, next_weight, next_bias, eps, branch_dtype)
    bare = y is None and residual_scale == 1.0
    r = x if bare else torch.empty(x.shape, dtype=x.dtype, device=dev)
    h = torch.empty(x.shape, dtype=bdt, device=dev) if next_norm else None
    stats = torch.empty((a.rows, 4), dtype=torch.float32, device=dev)
    a.stats = _addr(stats)
    _check(_lib.snack_residual_norm_forward(ctypes.byref(a), None if bare else _addr(r), _addr(h),
                                            _stream(stream, dev)))
    return r, h, stats


def _grad_rows(t, x, dtype, name):
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of type {dtype}")
    if t.shape != x.shape:
        raise ValueError(f"{name} {tuple(t.shape)} must have x's shape {tuple(x.shape)}")
    return _rows(t, name)[1]


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
    a, dev, bdt = _args(x, y, kind, post_norm, post_weight, post_bias, gate, residual_scale,
                        branch_scale, next_norm, next_weight, next_bias, eps, branch_dtype)
    if stats.dtype != torch.float32 or not stats.is_contiguous() or stats.numel() != 4 * a.rows:
        raise ValueError(f"stats must be {a.rows} x 4 contiguous float32")
    if dh is not None and not next_norm:
        raise ValueError("dh without next_norm")
    a.stats = _addr(stats)
    drs, dhs = _grad_rows(dr, x, x.dtype, "dr"), _grad_rows(dh, x, bdt, "dh")
    _same_device(x, dr, dh, stats)
    out = {"dx": torch.empty(x.shape, dtype=x.dtype, device=dev)}
    if y is not None:
        out["dy"] = torch.empty(x.shape, dtype=bdt, device=dev)
    for name, t in (("dgate", gate), ("dpost_weight", post_weight), ("dpost_bias", post_bias),
                    ("dnext_weight", next_weight), ("dnext_bias", next_bias)):
        if t is not None:
            out[name] = torch.empty(t.shape, dtype=t.dtype, device=dev)
    g = _abi.NormGrads(_addr(dr), _addr(dh), drs, dhs,
                       *[_addr(out.get(k)) for k in ("dx", "dy", "dgate", "dpost_weight",
                                                     "dpost_bias", "dnext_weight", "dnext_bias")])
    ws = torch.empty(_lib.snack_residual_norm_workspace(ctypes.byref(a)), dtype=torch.uint8,
                     device=dev)
    _record(ws, stream)
    _check(_lib.snack_residual_norm_backward(ctypes.byref(a), ctypes.byref(g), ws.data_ptr(),
                                             _stream(stream, dev)))
    return out


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
