"""Attention, forward and backward; the probabilities are never stored.

    out[i] = sum_j M[i, j] * softmax_j(scale * q[i] . k[j]) * v[j]

q is [sequences, tokens, heads, d], k and v [sequences, tokens, key heads, d]
(any strides, the last dimension contiguous); heads is a multiple of the key
heads.  With ``causal`` query i of nq sees the keys j <= i + nk - nq.  A
query that sees nothing gets zeros.

Sequences of unlike lengths: padded, with ``q_lengths`` / ``k_lengths``
(int32, one for each sequence; what lies behind is neither read nor seen, and
results there are zero), or packed end to end, q [tokens, heads, d] with
``q_offsets`` and k, v [tokens, key heads, d] with ``k_offsets`` (int32
[sequences + 1]).  All four lie on the device and are not read by the host.
A decode step over caches: q [sequences, 1, heads, d], k and v the whole
caches, ``k_lengths`` their fill, the new token included.

``dropout`` zeroes probabilities (M, a function of ``seed`` and the place:
the mask is made again in the backward pass).  ``seed`` is a number, or one
int64 on the device that is read when the kernels run: a captured graph
draws new masks where it also changes that tensor.
"""

from __future__ import annotations

import ctypes

import torch

from . import _check, _dense, _lib, _raw_stream, _stream
from ._autograd import first_derivative


def snack_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                            causal: bool = True, scale: float | None = None, q_offsets=None,
                            k_offsets=None, q_lengths=None, k_lengths=None, dropout: float = 0.0,
                            seed=0, stream=None):
    """(out, lse): out of q's shape, contiguous; lse float32 [heads, sequences, tokens]
    (ragged: [heads, tokens]), the log of each row's sum, -inf where it sees nothing.
    scale None: 1 / sqrt(d)."""
    return _dense.attention_forward(q, k, v, causal, scale, q_offsets, k_offsets, q_lengths,
                                    k_lengths, dropout, seed, _raw_stream(stream))


def snack_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                             v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, *,
                             causal: bool = True, scale: float | None = None, q_offsets=None,
                             k_offsets=None, q_lengths=None, k_lengths=None,
                             dropout: float = 0.0, seed=0, dq=None, dk=None, dv=None,
                             need_dq: bool = True, need_dkv: bool = True, stream=None):
    """(dq, dk, dv) from the forward call's out and lse and its options; None
    for what is not needed.  Tensors given as dq, dk, dv (any strides, no
    overlap) are overwritten and returned."""
    return _dense.attention_backward(dout, q, k, v, out, lse, causal, scale, q_offsets, k_offsets,
                                     q_lengths, k_lengths, dropout, seed, dq, dk, dv, need_dq,
                                     need_dkv, _raw_stream(stream))


def snack_attention_error(stream=None) -> bool:
    """Read and clear the current device's flag: True if a kernel of an attention call gave
    up a bounded wait since the last read (its block's results are then NaN).  Synchronises."""
    flag = ctypes.c_int()
    _check(_lib.snack_attention_error(ctypes.byref(flag), _stream(stream)))
    return bool(flag.value)


def snack_debug_attention_polls(polls: int) -> None:
    """Test hook: waits of attention kernels launched from now on give up after so many polls
    (negative: the usual limit)."""
    _lib.snack_debug_attention_polls(int(polls))


def _rows_contiguous(t):
    return t if t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


class _AttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, opts):
        out, lse = snack_attention_forward(q, k, v, **opts)
        ctx.names = [n for n, t in opts.items() if isinstance(t, torch.Tensor)]
        ctx.opts = {n: t for n, t in opts.items() if n not in ctx.names}
        ctx.save_for_backward(q, k, v, out, lse, *(opts[n] for n in ctx.names))
        return out

    @staticmethod
    @first_derivative
    def backward(ctx, dout):
        q, k, v, out, lse, *rest = ctx.saved_tensors
        need = ctx.needs_input_grad
        dq, dk, dv = snack_attention_backward(
            _rows_contiguous(dout), q, k, v, out, lse, need_dq=need[0], need_dkv=need[1] or need[2],
            **ctx.opts, **dict(zip(ctx.names, rest)))
        return dq, dk if need[1] else None, dv if need[2] else None, None


def snack_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, **opts) -> torch.Tensor:
    """out with gradients; the options of snack_attention_forward."""
    return _AttentionFunction.apply(q, k, v, opts)


def _split(qkv, heads, key_heads, ragged):
    width = qkv.shape[-1]
    if qkv.dim() != (2 if ragged else 3):
        raise ValueError("qkv must be [sequences, tokens, width], or [tokens, width] with q_offsets")
    if heads < 1 or key_heads < 1 or width % (heads + 2 * key_heads):
        raise ValueError(f"a width of {width} does not hold {heads} heads and twice {key_heads} key heads")
    d = width // (heads + 2 * key_heads)
    parts = qkv.split([heads * d, key_heads * d, key_heads * d], dim=-1)
    return tuple(t.unflatten(-1, (-1, d)) for t in parts)


_unsafe_view = torch.ops.aten._unsafe_view.default


class _PackedAttentionFunction(torch.autograd.Function):
    """The same on parts of one tensor, whose gradient is written in one piece."""

    @staticmethod
    def forward(ctx, qkv, heads, key_heads, opts):
        ragged = opts.get("q_offsets") is not None
        q, k, v = _split(qkv, heads, key_heads, ragged)
        out, lse = snack_attention_forward(q, k, v, **opts)
        # the same memory as a tensor that is nothing's view: a caller may write to it
        out = _unsafe_view(out, (*qkv.shape[:-1], heads * q.shape[-1]))
        ctx.shape = heads, key_heads, ragged
        ctx.names = [n for n, t in opts.items() if isinstance(t, torch.Tensor)]
        ctx.opts = {n: t for n, t in opts.items() if n not in ctx.names}
        ctx.save_for_backward(qkv, out, lse, *(opts[n] for n in ctx.names))
        return out

    @staticmethod
    @first_derivative
    def backward(ctx, dout):
        qkv, out, lse, *rest = ctx.saved_tensors
        q, k, v = _split(qkv, *ctx.shape)
        grad = torch.empty(qkv.shape, dtype=qkv.dtype, device=qkv.device)
        dq, dk, dv = _split(grad, *ctx.shape)
        snack_attention_backward(_rows_contiguous(dout).view(q.shape), q, k, v, out.view(q.shape), lse,
                                 dq=dq, dk=dk, dv=dv, **ctx.opts, **dict(zip(ctx.names, rest)))
        return grad, None, None, None


def snack_packed_attention(qkv: torch.Tensor, heads: int, key_heads: int | None = None, *,
                           offsets=None, lengths=None, **opts) -> torch.Tensor:
    """Self-attention of a projection's output [sequences, tokens, (heads + 2 * key_heads) * d]
    (or [tokens, ...] with ``offsets``), which holds every token's queries, then
    its keys, then its values; returns [..., heads * d], with gradients."""
    return _PackedAttentionFunction.apply(
        qkv, heads, heads if key_heads is None else key_heads,
        dict(opts, q_offsets=offsets, k_offsets=offsets, q_lengths=lengths, k_lengths=lengths))
