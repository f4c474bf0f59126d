"""The dense operators' C ABI, called through ctypes: what the Python binding never asks for."""

import ctypes

import torch

i64, i32, f32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p
TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
GATE = {None: 0, "channel": 1, "token": 2, "sequence": 3, "full": 4}
INVALID_ARG = 1


class NormArgs(ctypes.Structure):
    _fields_ = [("rows", i64), ("width", i64), ("group_rows", i64), ("norm_kind", i32),
                ("post_norm", i32), ("next_norm", i32), ("gate_kind", i32), ("stream_type", i32),
                ("branch_type", i32), ("param_type", i32), ("reserved", i32),
                ("residual_scale", f32), ("branch_scale", f32), ("eps", f32), ("reserved_f", f32),
                ("x", vp), ("y", vp), ("gate", vp), ("x_stride", i64), ("y_stride", i64),
                ("gate_stride", i64), ("post_weight", vp), ("post_bias", vp), ("next_weight", vp),
                ("next_bias", vp), ("stats", vp)]


class NormGrads(ctypes.Structure):
    _fields_ = [("dr", vp), ("dh", vp), ("dr_stride", i64), ("dh_stride", i64), ("dx", vp),
                ("dy", vp), ("dgate", vp), ("dpost_weight", vp), ("dpost_bias", vp),
                ("dnext_weight", vp), ("dnext_bias", vp)]


def lib():
    from coo_spmm_sparse_gb300 import _abi
    return _abi.load()


def ptr(t):
    return None if t is None else t.data_ptr()


def norm_args(x, y, stats, kind="rms", gate=None, gate_kind=None, group_rows=0, post_norm=0,
              next_norm=1, residual_scale=1.0, branch_scale=1.0, eps=1e-5, **params):
    """Arguments for contiguous x, y [rows][width]; params: post_weight, ... (float32)."""
    rows, width = x.shape
    return NormArgs(rows=rows, width=width, group_rows=group_rows,
                    norm_kind={"layer": 0, "rms": 1}[kind], post_norm=post_norm,
                    next_norm=next_norm, gate_kind=GATE[gate_kind], stream_type=TYPE[x.dtype],
                    branch_type=TYPE[x.dtype if y is None else y.dtype], param_type=0,
                    residual_scale=residual_scale, branch_scale=branch_scale, eps=eps, x=ptr(x),
                    y=ptr(y), gate=ptr(gate), x_stride=width, y_stride=width, gate_stride=width,
                    stats=ptr(stats), **{k: ptr(v) for k, v in params.items()})


def norm_forward(a, r, h, stream=None):
    return lib().snack_residual_norm_forward(ctypes.byref(a), ptr(r), ptr(h), stream)


def norm_backward(a, stream=None, **grads):
    """grads: contiguous tensors by the names of NormGrads' pointers."""
    g = NormGrads(dr_stride=a.width, dh_stride=a.width, **{k: ptr(v) for k, v in grads.items()})
    ws = torch.empty(lib().snack_residual_norm_workspace(ctypes.byref(a)), dtype=torch.uint8,
                     device="cuda")
    return lib().snack_residual_norm_backward(ctypes.byref(a), ctypes.byref(g), ws.data_ptr(),
                                              stream)
