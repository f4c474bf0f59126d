"""What the attention's and dropout's C calls refuse, before anything reaches a device (no GPU needed)."""

import ctypes

import pytest

i64, i32, f32, u64, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_uint64, ctypes.c_void_p
OK, INVALID, UNSUPPORTED = 0, 1, 6
FAKE = 1 << 20  # an address that is never read


class Args(ctypes.Structure):
    _fields_ = [("sequences", i64), ("q_tokens", i64), ("k_tokens", i64), ("heads", i32), ("key_heads", i32),
                ("head_size", i32), ("type", i32), ("causal", i32), ("scale", f32), ("dropout", f32),
                ("reserved", i32), ("seed", u64), ("seed_at", vp), ("q", vp), ("k", vp), ("v", vp),
                ("q_stride", i64 * 3), ("k_stride", i64 * 3), ("v_stride", i64 * 3), ("q_offsets", vp),
                ("k_offsets", vp), ("q_lengths", vp), ("k_lengths", vp)]


class Grads(ctypes.Structure):
    _fields_ = [("dout", vp), ("out", vp), ("lse", vp), ("dq", vp), ("dk", vp), ("dv", vp),
                ("dout_stride", i64 * 3), ("out_stride", i64 * 3), ("dq_stride", i64 * 3),
                ("dk_stride", i64 * 3), ("dv_stride", i64 * 3)]


def lib():
    from coo_spmm_sparse_gb300 import _abi
    return _abi.load()


def args(**change):
    base = dict(sequences=2, q_tokens=5, k_tokens=7, heads=4, key_heads=2, head_size=64, type=0, causal=1,
                scale=0.1, q=FAKE, k=FAKE, v=FAKE)
    return Args(**{**base, **change})


def forward(a):
    stride = (i64 * 3)(1280, 256, 64)
    return lib().snack_attention_forward(ctypes.byref(a), FAKE, stride, FAKE, FAKE, None)


@pytest.mark.parametrize("change,status", [
    (dict(type=3), INVALID), (dict(head_size=0), INVALID), (dict(head_size=129), INVALID),
    (dict(heads=3), INVALID), (dict(key_heads=0), INVALID), (dict(heads=0), INVALID), (dict(heads=-4), INVALID),
    (dict(sequences=-1), INVALID), (dict(q_tokens=-1), INVALID), (dict(k_tokens=-1), INVALID),
    (dict(causal=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(dropout=1.0), INVALID), (dict(dropout=-0.5), INVALID), (dict(dropout=float("nan")), INVALID),
    (dict(dropout=1 - 2.0 ** -18), INVALID), (dict(q_offsets=FAKE, q_lengths=FAKE), INVALID),
    (dict(k_offsets=FAKE, k_lengths=FAKE), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(q_stride=(i64 * 3)(1, -1, 1)), INVALID),
    (dict(k_stride=(i64 * 3)(-1, 1, 1)), INVALID), (dict(v_stride=(i64 * 3)(1, 1, -1)), INVALID),
    (dict(q_tokens=2 ** 31), UNSUPPORTED), (dict(k_tokens=2 ** 31), UNSUPPORTED),
    (dict(q_tokens=2 ** 30, heads=4), UNSUPPORTED), (dict(sequences=2 ** 25), UNSUPPORTED),
    (dict(sequences=2 ** 16 + 1, q_offsets=FAKE), UNSUPPORTED), (dict(sequences=2 ** 16 + 1, k_offsets=FAKE), UNSUPPORTED),
    (dict(sequences=2 ** 16, q_offsets=FAKE, heads=2 ** 16, key_heads=1), UNSUPPORTED),
    (dict(heads=2 ** 17, key_heads=2), UNSUPPORTED), (dict(sequences=2 ** 20, q_tokens=2 ** 20), UNSUPPORTED),
    (dict(sequences=2 ** 12, q_tokens=2 ** 20, dropout=0.1), UNSUPPORTED),
    (dict(sequences=2 ** 24, q_tokens=2 ** 31 - 8192, heads=2 ** 16, key_heads=2 ** 16), UNSUPPORTED),
    (dict(sequences=2 ** 24, k_tokens=2 ** 31 - 8192, heads=2 ** 16, key_heads=2 ** 16), UNSUPPORTED),
])
def test_attention_refuses(change, status):
    a = args(**change)
    assert forward(a) == status
    assert lib().snack_last_error(None)
    assert lib().snack_attention_backward(ctypes.byref(a), ctypes.byref(Grads()), FAKE, None) == status
    assert lib().snack_attention_forward_workspace(ctypes.byref(a)) == 0
    assert lib().snack_attention_backward_workspace(ctypes.byref(a)) == 0


def test_attention_needs_its_results():
    a, stride = args(), (i64 * 3)(1280, 256, 64)
    call = lib().snack_attention_forward
    assert call(None, FAKE, stride, FAKE, FAKE, None) == INVALID
    assert call(ctypes.byref(a), None, stride, FAKE, FAKE, None) == INVALID
    assert call(ctypes.byref(a), FAKE, None, FAKE, FAKE, None) == INVALID
    assert call(ctypes.byref(a), FAKE, stride, None, FAKE, None) == INVALID
    assert call(ctypes.byref(args(sequences=0)), None, None, None, None, None) == OK
    back = lib().snack_attention_backward
    full = dict(dout=FAKE, out=FAKE, lse=FAKE)
    assert back(ctypes.byref(a), None, FAKE, None) == INVALID
    assert back(ctypes.byref(a), ctypes.byref(Grads(**full)), None, None) == INVALID
    assert back(ctypes.byref(a), ctypes.byref(Grads(**full)), FAKE + 8, None) == INVALID
    for missing in full:
        assert back(ctypes.byref(a), ctypes.byref(Grads(**{**full, missing: None})), FAKE, None) == INVALID


@pytest.mark.parametrize("n,x,x_type,y,y_type,p,status", [
    (-1, FAKE, 0, FAKE, 0, 0.1, INVALID), (4, None, 0, FAKE, 0, 0.1, INVALID), (4, FAKE, 0, None, 0, 0.1, INVALID),
    (4, FAKE, 3, FAKE, 0, 0.1, INVALID), (4, FAKE, 0, FAKE, -1, 0.1, INVALID), (4, FAKE, 0, FAKE, 0, 1.0, INVALID),
    (4, FAKE, 0, FAKE, 0, float("nan"), INVALID), (2 ** 41, FAKE, 0, FAKE, 0, 0.1, UNSUPPORTED),
    (0, None, 0, None, 0, 0.1, OK),
])
def test_dropout_refuses(n, x, x_type, y, y_type, p, status):
    assert lib().snack_dropout(n, x, x_type, None, y, y_type, p, 0, None, None) == status
