"""Low-rank adapters of many requests at once beside one projection.

Request i owns the tokens offsets[i] .. offsets[i+1]-1 of X and names adapter
n = adapter[i] (-1: none).  For each of its tokens

    H[t] = A[n] X[t],    Y[t] += scale[n] * B[n] H[t]

Y arrives with the shared projection's output (``snack_forward``) and leaves
with the adapters' part added.  ``SnackAdapters`` keeps the weights of the
adapters of one projection and carries the gradients.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _abi, _addr, _check, _dense_type, _lib, _rows, _same_device, _stream
from .grad_clip import _record


def _args(X, A, B, offsets, adapter, scale):
    kind = _dense_type(X, "X")
    for t, name in ((A, "A"), (B, "B")):
        if _dense_type(t, name) != kind:
            raise TypeError(f"{name} must have X's type")
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with three dimensions")
    n, rank, inp = A.shape
    out = B.shape[1]
    if B.shape[0] != n or B.shape[2] != rank:
        raise ValueError(f"A is [adapters][rank][in] {tuple(A.shape)}, so B must be "
                         f"[{n}][out][{rank}], got {tuple(B.shape)}")
    if X.dim() < 1 or X.shape[-1] != inp:
        raise ValueError(f"X must be [..., {inp}], got {tuple(X.shape)}")
    for t, name in ((offsets, "offsets"), (adapter, "adapter")):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.int32
                and t.dim() == 1 and t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous CUDA int32 vector")
    if offsets.numel() != adapter.numel() + 1:
        raise ValueError("offsets must have one element more than adapter")
    uniform, sp = 1.0, None
    if isinstance(scale, torch.Tensor):
        if scale.dtype != torch.float32 or not scale.is_contiguous() or scale.numel() != n:
            raise ValueError(f"scale must be a number or {n} contiguous float32")
        sp = scale
    else:
        uniform = float(scale)
    dev = _same_device(X, A, B, offsets, adapter, sp)
    rows, stride = _rows(X, "X")
    a = _abi.AdapterArgs(rows, adapter.numel(), n, inp, out, rank, kind, uniform, _addr(X),
                         _addr(A), _addr(B), stride, _addr(offsets), _addr(adapter), _addr(sp))
    return a, dev


def _like(t, X, width, rows, name):
    """Row stride of t, which must be X's type with `width` columns and as many rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != X.dtype:
        raise TypeError(f"{name} must be a CUDA tensor of X's type")
    if t.shape[-1] != width:
        raise ValueError(f"{name} must be [..., {width}], got {tuple(t.shape)}")
    n, stride = _rows(t, name)
    if n != rows:
        raise ValueError(f"{name} has {n} rows, X has {rows}")
    return stride


def snack_adapter_forward(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                          offsets: torch.Tensor, adapter: torch.Tensor, scale, Y: torch.Tensor,
                          H: torch.Tensor | None = None, stream=None):
    """Add the adapters' part to Y in place; returns (Y, H) with H [tokens][rank] float32.

    X [..., in] and Y [..., out] may have strided rows; A [adapters][rank][in],
    B [adapters][out][rank]; offsets [requests + 1] and adapter [requests] int32
    on the device (not read by the host); scale a number or float32 [adapters]."""
    a, dev = _args(X, A, B, offsets, adapter, scale)
    ys = _like(Y, X, a.out, a.tokens, "Y")
    if H is None:
        H = torch.empty((a.tokens, a.rank), dtype=torch.float32, device=dev)
    elif H.dtype != torch.float32 or not H.is_contiguous() or H.numel() != a.tokens * a.rank:
        raise ValueError(f"H must be {a.tokens} x {a.rank} contiguous float32")
    _same_device(X, Y, H)
    ws = torch.empty(_lib.snack_adapter_forward_workspace(ctypes.byref(a)), dtype=torch.uint8,
                     device=dev)
    _record(ws, stream)
    _check(_lib.snack_adapter_forward(ctypes.byref(a), _addr(Y), ys, _addr(H), ws.data_ptr(),
                                      _stream(stream, dev)))
    return Y, H


def snack_adapter_backward(X: torch.Tensor, dY: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                           offsets: torch.Tensor, adapter: torch.Tensor, scale, H: torch.Tensor,
                           dX: torch.Tensor | None = None, need_dx: bool = True,
                           need_dw: bool = True, stream=None):
    """(dX, dA, dB) of the adapters' part of Y.  dX is added to in place where
    it is given (the projection's own input gradient), else started from
    zeros; dA and dB have the shapes of A and B."""
    a, dev = _args(X, A, B, offsets, adapter, scale)
    dys = _like(dY, X, a.out, a.tokens, "dY")
    if H.dtype != torch.float32 or not H.is_contiguous() or H.numel() != a.tokens * a.rank:
        raise ValueError(f"H must be {a.tokens} x {a.rank} contiguous float32")
    dxs = a.inp
    if not need_dx:
        dX = None
    elif dX is None:
        dX = torch.zeros(X.shape, dtype=X.dtype, device=dev)
    else:
        dxs = _like(dX, X, a.inp, a.tokens, "dX")
    dA = torch.empty_like(A) if need_dw else None
    dB = torch.empty_like(B) if need_dw else None
    _same_device(X, dY, H, dX)
    ws = torch.empty(_lib.snack_adapter_backward_workspace(ctypes.byref(a)), dtype=torch.uint8,
                     device=dev)
    _record(ws, stream)
    _check(_lib.snack_adapter_backward(ctypes.byref(a), _addr(dY), dys, _addr(H), _addr(dX), dxs,
                                       _addr(dA), _addr(dB), ws.data_ptr(), _stream(stream, dev)))
    return dX, dA, dB


class _AdapterFunction(torch.autograd.Function):
    """Y of the projection with the adapters' part added in place."""

    @staticmethod
    def forward(ctx, X, Y, A, B, offsets, adapter, scale):
        _, H = snack_adapter_forward(X, A, B, offsets, adapter, scale, Y)
        ctx.mark_dirty(Y)
        ctx.scale = scale
        ctx.save_for_backward(X, A, B, offsets, adapter, H)
        return Y

    @staticmethod
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
    output y (in place) and returns it.  ``scale`` is alpha / rank."""

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
