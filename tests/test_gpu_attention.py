"""Attention and its gradients against a 64-bit evaluation of their definition
(bounds in attention_ref.py), the gradients also against differences."""

import pytest
import torch

import attention_ref
from attention_ref import assert_within

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


def rnd(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check(q, k, v, dout, **opts):
    import coo_spmm_sparse_gb300 as sn
    out, lse = sn.snack_attention_forward(q, k, v, **opts)
    got = {"out": out, "lse": lse}
    if dout is not None:
        got["dq"], got["dk"], got["dv"] = sn.snack_attention_backward(dout, q, k, v, out, lse, **opts)
    torch.cuda.synchronize()
    assert_within(got, attention_ref.attention(q, k, v, dout=dout, **opts))
    return got


def dense(start, n, nq, nk, heads, key_heads, d, dtype, **opts):
    g = gen(start)
    q, dout = (rnd(g, (n, nq, heads, d), dtype) for _ in range(2))
    k, v = (rnd(g, (n, nk, key_heads, d), dtype) for _ in range(2))
    return check(q, k, v, dout, **opts)


def offsets(*lengths):
    return torch.tensor([0, *lengths], device="cuda").cumsum(0).to(torch.int32)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 2), (2, 1), (1, 257), (3, 64), (16, 16), (17, 33), (64, 64),
                                   (65, 127), (128, 128), (129, 129), (255, 300), (300, 40), (513, 513)])
def test_every_length(dtype, causal, nq, nk):
    dense(nq * 1000 + nk, 2, nq, nk, 4, 2, 64, dtype, causal=causal)
    dense(nq * 1000 + nk, 1, nq, nk, 3, 3, 128, dtype, causal=causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [1, 2, 3, 7, 8, 16, 31, 32, 40, 63, 64, 65, 72, 80, 96, 100, 112, 127, 128])
def test_every_head_size(dtype, d):
    dense(d, 2, 70, 90, 4, 2, d, dtype)
    dense(d, 1, 200, 200, 2, 2, d, dtype, dropout=0.2, seed=d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,key_heads", [(1, 1), (3, 1), (5, 5), (6, 2), (8, 1), (12, 4), (16, 2), (32, 1)])
def test_shared_heads(dtype, heads, key_heads):
    dense(heads, 2, 133, 133, heads, key_heads, 64, dtype)
    dense(heads, 3, 1, 500, heads, key_heads, 128, dtype)
    dense(heads, 2, 7, 1030, heads, key_heads, 80, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,length,heads,key_heads,d", [(2, 1024, 40, 20, 64), (1, 2100, 24, 8, 128),
                                                        (3, 1500, 16, 16, 80), (1, 4097, 8, 1, 64)])
def test_long_sequences_that_fill_the_gpu(dtype, n, length, heads, key_heads, d):
    dense(length, n, length, length, heads, key_heads, d, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [1, 33, 40, 63, 64, 100, 128])
@pytest.mark.parametrize("dropout", [0.0, 0.2])
def test_tensors_that_cannot_be_copied_as_they_lie(dtype, d, dropout):
    """Odd head sizes, addresses off 16 bytes and heads before tokens, at sizes where the operands
    are made in float16 first (32-bit floats from 4e6 query rows times keys on)."""
    g = gen(d)
    n, length = 2, 777
    q, dout = (rnd(g, (n, length, 6, d + 1), dtype)[..., 1:] for _ in range(2))
    k = rnd(g, (n, 3, length, d), dtype).transpose(1, 2)
    v = rnd(g, (n, length, 1, d), dtype).expand(n, length, 3, d)
    check(q, k, v, dout, dropout=dropout, seed=d)
    check(q, k, v, dout.contiguous(), causal=False, k_lengths=ints(777, 300))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,q,k,d", [(1, 130, 9000, 64), (2, 200, 6001, 128), (1, 300, 2100, 80), (3, 64, 20000, 64)])
def test_many_queries_over_keys_in_parts(dtype, n, q, k, d):
    g = gen(k)
    fill = torch.randint(q - 10, k + 1, (n,), generator=g, device="cuda").to(torch.int32)
    args = [rnd(g, (n, q, 8, d), dtype), rnd(g, (n, k, 2, d), dtype), rnd(g, (n, k, 2, d), dtype)]
    for t in args[1:]:
        for i in range(n):
            t[i, fill[i]:] = float("nan")
    check(*args, None, k_lengths=fill)
    check(*args, None, k_lengths=fill, causal=False, dropout=0.3, seed=11)
    check(*args, rnd(g, (n, q, 8, d), dtype), k_lengths=fill)


def test_operands_of_every_magnitude():
    """Tensors far from one another and from 1, channels and tokens far from their tensor's largest."""
    for dtype in (F32, BF16):
        for scales in ((1e-9, 1e9, 1e5), (1e6, 1e-6, 1e-12), (1.0, 1.0, 1e20)):
            g = gen(3)
            q, k, v = (rnd(g, (1, 1100, 4, 64), dtype, s) for s in scales)
            v[..., ::7] *= 1e-3
            q[:, ::5] *= 1e-2
            check(q, k, v, rnd(g, (1, 1100, 4, 64), dtype, 1e-6))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,q,k", [(1, 1, 32768), (2, 1, 5000), (4, 2, 3001), (40, 1, 700), (1, 19, 9000)])
def test_few_queries_over_long_caches(dtype, n, q, k):
    g = gen(k)
    cache_k, cache_v = (rnd(g, (n, k, 2, 128), dtype) for _ in range(2))
    fill = torch.randint(q, k + 1, (n,), generator=g, device="cuda").to(torch.int32)
    for i in range(n):  # what lies behind a cache's fill is not read
        cache_k[i, fill[i]:] = float("nan")
        cache_v[i, fill[i]:] = float("inf")
    check(rnd(g, (n, q, 8, 128), dtype), cache_k, cache_v, None, k_lengths=fill)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("dropout", [0.0, 0.3])
def test_ragged(dtype, d, dropout):
    g = gen(d)
    off = offsets(5, 0, 1, 300, 64, 129, 0, 700, 128)
    total = int(off[-1])
    qkv = rnd(g, (total, 12 * d), dtype)
    q, k, v = (t.unflatten(-1, (-1, d)) for t in qkv.split([8 * d, 2 * d, 2 * d], dim=-1))
    check(q, k, v, rnd(g, (total, 8, d), dtype), q_offsets=off, k_offsets=off, dropout=dropout, seed=3)


@pytest.mark.parametrize("dtype", TYPES)
def test_ragged_to_other_sequences(dtype):
    g = gen(1)
    qo, ko = offsets(7, 300, 0, 40, 130), offsets(200, 31, 9, 0, 140)
    for causal in (True, False):
        check(rnd(g, (477, 4, 64), dtype), rnd(g, (380, 2, 64), dtype), rnd(g, (380, 2, 64), dtype),
              rnd(g, (477, 4, 64), dtype), q_offsets=qo, k_offsets=ko, causal=causal)


@pytest.mark.parametrize("dtype", TYPES)
def test_new_tokens_packed_over_dense_caches(dtype):
    g = gen(2)
    check(rnd(g, (150, 4, 64), dtype), rnd(g, (3, 200, 2, 64), dtype), rnd(g, (3, 200, 2, 64), dtype),
          rnd(g, (150, 4, 64), dtype), q_offsets=offsets(100, 1, 49), k_lengths=ints(180, 200, 60))
    check(rnd(g, (3, 20, 4, 64), dtype), rnd(g, (150, 2, 64), dtype), rnd(g, (150, 2, 64), dtype),
          rnd(g, (3, 20, 4, 64), dtype), k_offsets=offsets(100, 1, 49))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_outside_every_sequence(dtype, d):
    g = gen(3)
    off = ints(10, 150, 290)
    q, k, v, dout = (rnd(g, (500, 2, d), dtype) for _ in range(4))
    for t in (q, k, v, dout):
        t[:10] = float("nan")
        t[290:] = float("nan")
    got = check(q, k, v, dout, q_offsets=off, k_offsets=off)
    for name in ("out", "dq", "dk", "dv"):
        assert not got[name][:10].any() and not got[name][290:].any(), name
    none = check(q, k, v, dout, q_offsets=ints(0), k_offsets=ints(0))
    for name in ("out", "dq", "dk", "dv"):
        assert not none[name].any(), name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,length,d", [(3, 100, 64), (3, 300, 128), (24, 700, 64)])
def test_padding_is_neither_read_nor_seen(dtype, n, length, d):
    g = gen(4)
    q, k, v, dout = (rnd(g, (n, length, 8, d), dtype) for _ in range(4))
    fill = torch.randint(0, length + 1, (n,), generator=g, device="cuda").to(torch.int32)
    fill[0] = 0
    for t in (q, k, v, dout):
        for i in range(n):
            t[i, fill[i]:] = float("nan")
    got = check(q, k, v, dout, q_lengths=fill, k_lengths=fill, dropout=0.1, seed=2 ** 63 + 5)
    for name in ("out", "dq", "dk", "dv"):
        for i in range(n):
            assert not got[name][i, fill[i]:].any(), name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length,d", [(37, 64), (300, 128), (513, 64)])
def test_strides(dtype, length, d):
    g = gen(5)

    def heads_first(h):
        return rnd(g, (2, h, length, d), dtype).transpose(1, 2)

    check(heads_first(6), heads_first(2), heads_first(2), heads_first(6))
    # one key head for all by a stride of zero, and rows that begin off a vector
    k = rnd(g, (2, length, 1, d), dtype).expand(2, length, 6, d)
    v = rnd(g, (2, length, 1, d + 3), dtype)[..., 3:].expand(2, length, 6, d)
    wide = rnd(g, (2, length, 6, d + 1), dtype)
    check(wide[..., 1:], k, v, wide[..., :-1])
    big = rnd(g, (2, length, 6, 2 * d), dtype)
    check(big[..., :d], big[:, :, :3, d:], big[:, :, 3:, d:], big[..., d:])


@pytest.mark.parametrize("dtype", TYPES)
def test_results_into_strided_tensors(dtype):
    import coo_spmm_sparse_gb300 as sn
    g = gen(6)
    for d, length in ((64, 50), (128, 400), (33, 60)):
        q, k, v, dout = (rnd(g, (2, length, 4, d), dtype) for _ in range(4))
        out, lse = sn.snack_attention_forward(q, k, v)
        want = sn.snack_attention_backward(dout, q, k, v, out, lse)
        room = torch.full((2, length, 3, 4, d + 1), 7.0, device="cuda", dtype=dtype)
        views = [room[:, :, i, :, 1:] for i in range(3)]
        got = sn.snack_attention_backward(dout, q, k, v, out, lse, dq=views[0], dk=views[1], dv=views[2])
        for a, b in zip(got, want):
            assert_within({"x": a}, {"x": (b.double(), 2.0 ** -6 * b.double().abs() + 1e-3)})
        assert (room[..., 0] == 7.0).all()
        only = sn.snack_attention_backward(dout, q, k, v, out, lse, need_dkv=False)
        assert only[1] is None and torch.equal(only[0], want[0])
        only = sn.snack_attention_backward(dout, q, k, v, out, lse, need_dq=False)
        assert only[0] is None and torch.equal(only[1], want[1]) and torch.equal(only[2], want[2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,nk", [(1, 300), (60, 60), (400, 400)])
def test_scores_of_every_size(dtype, nq, nk):
    """Scores of +-300, one key far above the others late in the row, negative and zero scales."""
    g = gen(7)
    q, dout = (rnd(g, (2, nq, 4, 64), dtype, 6.0) for _ in range(2))
    k, v = (rnd(g, (2, nk, 4, 64), dtype, 6.0) for _ in range(2))
    k[:, nk - nk // 3] *= 3.0
    check(q, k, v, dout)
    check(q, k, v, dout, scale=-0.2)
    check(q, k, v, dout, scale=0.0)
    check(q * 0, k, v, dout)


@pytest.mark.parametrize("dtype", TYPES)
def test_queries_that_see_one_key_move_no_score(dtype):
    """Softmax of one score is 1: dq and dk are exactly zero, not what two roundings leave."""
    import coo_spmm_sparse_gb300 as sn
    g = gen(18)
    for n, nq, room, opts in ((10, 1, 1, {}), (3, 300, 300, dict(causal=False)), (200, 70, 70, dict(causal=False))):
        q, dout = (rnd(g, (n, nq, 4, 64), dtype) for _ in range(2))
        k, v = (rnd(g, (n, room, 2, 64), dtype) for _ in range(2))
        o = dict(k_lengths=torch.ones(n, dtype=torch.int32, device="cuda"), dropout=0.2, seed=1, **opts)
        out, lse = sn.snack_attention_forward(q, k, v, **o)
        dq, dk, dv = sn.snack_attention_backward(dout, q, k, v, out, lse, **o)
        assert not dq.any() and not dk.any() and dv[:, 0].any()
    # the first query of a causal call, among others
    q, k, v, dout = (rnd(g, (2, 900, 4, 64), dtype) for _ in range(4))
    out, lse = sn.snack_attention_forward(q, k, v)
    dout[:, 1:] = 0
    dq, dk, dv = sn.snack_attention_backward(dout, q, k, v, out, lse)
    assert not dq[:, 0].any() and not dk.any()
    # its probability is exp(s - lse): off by a share 2 * 2^-18 * A + 2^-16 at most, A below 16 here
    share = 2.0 ** -13 + 2.0 ** -16 + attention_ref.U[dtype]
    assert ((dv[:, 0].double() - dout[:, 0].double()).abs() <= share * dout[:, 0].double().abs() + 1e-7).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n, nq, nk, heads, key_heads, d, causal", [
    (1, 2, 2, 8, 8, 64, True), (2, 32, 32, 2, 1, 48, True), (3, 5, 9, 4, 2, 65, False),
    (8, 16, 16, 24, 12, 128, True),   # rows * heads * d = 393216
    (8, 1024, 2, 12, 12, 64, True)])  # most rows see no key
def test_gradients_of_few_keys_are_free_of_the_rounding_of_out(dtype, n, nq, nk, heads, key_heads, d, causal):
    import coo_spmm_sparse_gb300 as sn
    g = gen(19)
    q, dout = (rnd(g, (n, nq, heads, d), dtype) for _ in range(2))
    k, v = (rnd(g, (n, nk, key_heads, d), dtype) for _ in range(2))
    opts = dict(causal=causal, dropout=0.2, seed=3)
    out, lse = sn.snack_attention_forward(q, k, v, **opts)
    want = sn.snack_attention_backward(dout, q, k, v, out, lse, **opts)
    other = out * (1 + torch.finfo(dtype).eps)
    assert not torch.equal(other, out)
    got = sn.snack_attention_backward(dout, q, k, v, other, lse, **opts)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_few_keys_on_both_sides_of_the_rule(dtype):
    g = gen(20)
    for n, length in ((2, 32), (2, 33), (8, 17), (300, 2)):
        q, dout = (rnd(g, (n, length, 24, 128), dtype) for _ in range(2))
        k, v = (rnd(g, (n, length, 12, 128), dtype) for _ in range(2))
        check(q, k, v, dout, dropout=0.2, seed=1)
    at = offsets(0, 3, 1, 12, 16)  # 32 tokens
    q, dout = (rnd(g, (32, 4, 72), dtype) for _ in range(2))
    k, v = (rnd(g, (32, 2, 72), dtype) for _ in range(2))
    check(q, k, v, dout, q_offsets=at, k_offsets=at)


def test_small_float16_gradients():
    """A loss that is a mean makes gradients that float16 only holds as subnormals."""
    g = gen(8)
    q, k, v = (rnd(g, (1, 700, 4, 64), F16) for _ in range(3))
    for std in (1e-3, 3e-5, 1000.0):
        check(q, k, v, rnd(g, (1, 700, 4, 64), F16, std), dropout=0.5, seed=1)
    check(q, k, v * 0, rnd(g, (1, 700, 4, 64), F16))


@pytest.mark.parametrize("dtype", TYPES)
def test_dropout_takes_its_mask_from_the_seed(dtype):
    import coo_spmm_sparse_gb300 as sn
    n, d = 96, 96
    q = torch.zeros(1, n, 2, d, device="cuda", dtype=dtype)
    v = torch.eye(n, d, device="cuda", dtype=dtype)[None, :, None].expand(1, n, 2, d)
    for p in (0.25, 1e-5, 65535 / 65536):
        out, _ = sn.snack_attention_forward(q, v, v, causal=False, dropout=p, seed=-3)
        row = torch.arange(n, device="cuda")[:, None] * 2 + torch.arange(2, device="cuda")
        M = attention_ref.mask_of(-3, row << 30, n, p)
        assert torch.equal(out[0] != 0, M != 0)
        assert torch.allclose(out[0].double(), M / n, rtol=2.0 ** -7)
    spot = [(5, 1, 17), (95, 0, 95), (0, 0, 0)]
    out, _ = sn.snack_attention_forward(q, v, v, causal=False, dropout=0.25, seed=77)
    for i, h, j in spot:
        bits = attention_ref.draw(77, ((i * 2 + h) << 30) + j // 4) >> (16 * (j % 4)) & 0xFFFF
        assert bool(out[0, i, h, j]) == (bits >= 16384)


@pytest.mark.parametrize("dropout", [0.0, 0.25])
@pytest.mark.parametrize("n,d,dtype", [(20, 16, F32), (150, 64, F32)])
def test_gradients_against_differences(n, d, dtype, dropout):
    """(f(x + h u) - f(x - h u)) / 2h of f = sum(out * dout): its own error is h^2 / 6 of
    the third derivative (scores and values of order one: below 1e-4 of the gradient's
    terms at h = 2^-6 over these sizes), and two roundings of f's terms over h."""
    import coo_spmm_sparse_gb300 as sn
    g = gen(9)
    x = [rnd(g, (1, n, 2, d), dtype, 0.5) for _ in range(3)]
    dout = rnd(g, (1, n, 2, d), dtype)
    opts = dict(dropout=dropout, seed=5)
    out, lse = sn.snack_attention_forward(*x, **opts)
    grads = sn.snack_attention_backward(dout, *x, out, lse, **opts)
    h = 2.0 ** -6
    for i in range(3):
        u = rnd(g, (1, n, 2, d), dtype)
        u /= u.norm()
        f = []
        for sign in (h, -h):
            y = [t + sign * u if j == i else t for j, t in enumerate(x)]
            f.append((sn.snack_attention_forward(*y, **opts)[0].double() * dout.double()).sum())
        want = float((f[0] - f[1]) / (2 * h))
        got = float((grads[i].double() * u.double()).sum())
        terms = float((out.double() * dout.double()).abs().sum())
        size = float(grads[i].double().norm())
        assert abs(got - want) <= 1e-3 * size + 2e-6 * terms ** 0.5 / h, (i, got, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_again(dtype):
    import coo_spmm_sparse_gb300 as sn
    g = gen(10)
    for n, length, heads, key_heads, d in ((1, 256, 12, 12, 64), (2, 1000, 8, 2, 128)):
        q, dout = (rnd(g, (n, length, heads, d), dtype) for _ in range(2))
        k, v = (rnd(g, (n, length, key_heads, d), dtype) for _ in range(2))
        runs = []
        for _ in range(3):
            out, lse = sn.snack_attention_forward(q, k, v, dropout=0.1, seed=4)
            runs.append((out, lse, *sn.snack_attention_backward(dout, q, k, v, out, lse, dropout=0.1, seed=4)))
        for r in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("dtype", TYPES)
def test_autograd(dtype):
    import coo_spmm_sparse_gb300 as sn
    g = gen(11)
    q, k, v = (rnd(g, (2, 90, h, 64), dtype).requires_grad_() for h in (6, 3, 3))
    dout = rnd(g, (2, 90, 6, 64), dtype)
    out = sn.snack_attention(q, k, v, dropout=0.1, seed=9)
    out.backward(dout)
    o, lse = sn.snack_attention_forward(q.detach(), k.detach(), v.detach(), dropout=0.1, seed=9)
    want = sn.snack_attention_backward(dout, q.detach(), k.detach(), v.detach(), o, lse, dropout=0.1, seed=9)
    assert torch.equal(out.detach(), o)
    for t, w in zip((q, k, v), want):
        assert torch.equal(t.grad, w)
    # a gradient without strides of its own
    q.grad = None
    sn.snack_attention(q, k, v).sum().backward()
    o, lse = sn.snack_attention_forward(q.detach(), k.detach(), v.detach())
    assert torch.equal(q.grad, sn.snack_attention_backward(torch.ones_like(o), q.detach(), k.detach(),
                                                           v.detach(), o, lse)[0])
    (dq,) = torch.autograd.grad(sn.snack_attention(q, k, v).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        dq.sum().backward()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ragged", [False, True])
def test_packed_projection(dtype, ragged):
    import coo_spmm_sparse_gb300 as sn
    g = gen(12)
    d, H, Hk = 64, 6, 2
    qkv = rnd(g, (330, (H + 2 * Hk) * d) if ragged else (3, 110, (H + 2 * Hk) * d), dtype)
    opts = dict(offsets=offsets(100, 0, 230)) if ragged else dict(lengths=ints(110, 40, 0))
    dout = rnd(g, (*qkv.shape[:-1], H * d), dtype)
    a = qkv.clone().requires_grad_()
    out = sn.snack_packed_attention(a, H, Hk, dropout=0.2, seed=1, **opts)
    out.backward(dout)
    b = qkv.clone().requires_grad_()
    q, k, v = (t.unflatten(-1, (-1, d)) for t in b.split([H * d, Hk * d, Hk * d], dim=-1))
    names = ("q_offsets", "k_offsets") if ragged else ("q_lengths", "k_lengths")
    other = sn.snack_attention(q, k, v, dropout=0.2, seed=1, **{n: list(opts.values())[0] for n in names})
    other.flatten(-2).backward(dout)
    assert torch.equal(out, other.flatten(-2)) and torch.equal(a.grad, b.grad)
    for bad in ((H, 3), (0, 1), (H, 0)):
        with pytest.raises(ValueError):
            sn.snack_packed_attention(qkv, *bad, **opts)


def test_captured_calls_draw_again_when_their_seed_changes():
    import coo_spmm_sparse_gb300 as sn
    g = gen(13)
    q, k, v, dout = (rnd(g, (1, 200, 4, 64), BF16) for _ in range(4))
    seed = torch.tensor(100, device="cuda")

    def both():
        out, lse = sn.snack_attention_forward(q, k, v, dropout=0.5, seed=seed)
        return (out, *sn.snack_attention_backward(dout, q, k, v, out, lse, dropout=0.5, seed=seed))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = both()
        seed.add_(1)
    for step in range(3):
        graph.replay()
        out, lse = sn.snack_attention_forward(q, k, v, dropout=0.5, seed=100 + step)
        want = (out, *sn.snack_attention_backward(dout, q, k, v, out, lse, dropout=0.5, seed=100 + step))
        assert all(torch.equal(a, b) for a, b in zip(res, want))


@pytest.mark.parametrize("dtype", TYPES)
def test_calls_on_two_streams_and_in_two_graphs(dtype):
    """Two calls at once, each with its own workspace: the same results as alone."""
    import coo_spmm_sparse_gb300 as sn
    g = gen(16)
    sets = [[rnd(g, (2, 900, 6, 64), dtype) for _ in range(4)] for _ in range(2)]

    def both(q, k, v, dout):
        out, lse = sn.snack_attention_forward(q, k, v)
        return (out, *sn.snack_attention_backward(dout, q, k, v, out, lse))

    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(both(*s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    graphs, res = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            res.append(both(*s))
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not sn.snack_attention_error()


def test_a_given_stream():
    import coo_spmm_sparse_gb300 as sn
    g = gen(14)
    q, k, v = (rnd(g, (1, 1, 8, 128), BF16), *(rnd(g, (1, 9000, 2, 128), BF16) for _ in range(2)))
    want = sn.snack_attention_forward(q, k, v)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sn.snack_attention_forward(q, k, v, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_broken_offsets_touch_nothing_outside(dtype):
    import coo_spmm_sparse_gb300 as sn
    g = gen(15)
    room = rnd(g, (3, 400, 2, 64), dtype)
    keep = room.clone()
    q = room[1]
    off = ints(-5, 90, 40, 10 ** 9, 200)
    out, lse = sn.snack_attention_forward(q, q, q, q_offsets=off, k_offsets=off)
    big = torch.full((3, 400, 2, 64), 5.0, device="cuda", dtype=dtype)
    sn.snack_attention_backward(q, q, q, q, out, lse, q_offsets=off, k_offsets=off, dq=big[1], dk=torch.empty_like(q),
                                dv=torch.empty_like(q))
    fill = ints(10 ** 9, -3, 7)
    sn.snack_attention_forward(room, room, room, q_lengths=fill, k_lengths=fill)
    torch.cuda.synchronize()
    assert torch.equal(room, keep) and (big[0] == 5.0).all() and (big[2] == 5.0).all()


def test_nothing_to_do():
    import coo_spmm_sparse_gb300 as sn
    for shape, kshape in (((0, 5, 2, 64), (0, 5, 2, 64)), ((2, 0, 2, 64), (2, 5, 2, 64)), ((2, 5, 2, 64), (2, 0, 2, 64))):
        q, k = torch.ones(shape, device="cuda"), torch.ones(kshape, device="cuda")
        out, lse = sn.snack_attention_forward(q, k, k)
        dq, dk, dv = sn.snack_attention_backward(q, q, k, k, out, lse)
        assert out.shape == shape and not out.any() and not dq.any() and not dk.any() and not dv.any()
        assert (lse == -torch.inf).all()


def test_refusals():
    import coo_spmm_sparse_gb300 as sn
    t = lambda *s, dt=F32: torch.zeros(s, device="cuda", dtype=dt)  # noqa: E731
    q, k = t(2, 5, 4, 64), t(2, 7, 2, 64)
    f = sn.snack_attention_forward
    off, fill = ints(0, 3, 5), ints(1, 2)
    for err, args, opts in [
        (TypeError, (q.cpu(), k, k), {}), (TypeError, (q.double(), k, k), {}), (TypeError, (q, k.half(), k), {}),
        (TypeError, (q, k, k.half()), {}), (ValueError, (q, k, t(2, 8, 2, 64)), {}),
        (ValueError, (q[0], k, k), {}), (ValueError, (q, k[0], k[0]), {}),
        (ValueError, (q, t(3, 7, 2, 64), t(3, 7, 2, 64)), {}), (ValueError, (q, t(2, 7, 3, 64), t(2, 7, 3, 64)), {}),
        (ValueError, (q, t(2, 7, 2, 32), t(2, 7, 2, 32)), {}),
        (ValueError, (t(1, 5, 4, 129), t(1, 5, 4, 129), t(1, 5, 4, 129)), {}),
        (ValueError, (t(2, 5, 64, 4).transpose(2, 3), k, k), {}), (ValueError, (q, k, k), dict(scale=float("inf"))),
        (ValueError, (q, k, k), dict(dropout=1.0)), (ValueError, (q, k, k), dict(dropout=-0.1)),
        (ValueError, (q, k, k), dict(dropout=float("nan"))), (sn.SnackError, (q, k, k), dict(dropout=1 - 2.0 ** -18)),
        (ValueError, (q, k, k), dict(q_offsets=off)), (ValueError, (q[0], k, k), dict(q_offsets=off, q_lengths=fill)),
        (ValueError, (q, k, k), dict(k_lengths=ints(1))), (TypeError, (q, k, k), dict(k_lengths=fill.long())),
        (TypeError, (q, k, k), dict(k_lengths=fill.cpu())), (TypeError, (q, k, k), dict(dropout=0.1, seed=1.5)),
        (TypeError, (q, k, k), dict(dropout=0.1, seed=torch.tensor(1))),
        (TypeError, (q, k, k), dict(dropout=0.1, seed=torch.ones(2, device="cuda", dtype=torch.long))),
    ]:
        with pytest.raises(err):
            f(*args, **opts)
    out, lse = f(q, k, k)
    b = sn.snack_attention_backward
    for err, args, opts in [
        (ValueError, (q[:, :4], q, k, k, out, lse), {}), (TypeError, (q.half(), q, k, k, out, lse), {}),
        (ValueError, (q, q, k, k, out[:, :4], lse), {}), (ValueError, (q, q, k, k, out, lse[:2]), {}),
        (ValueError, (q, q, k, k, out, lse.transpose(0, 1)), {}), (ValueError, (q, q, k, k, out, lse.half()), {}),
        (ValueError, (q, q, k, k, out, lse), dict(dq=k)), (TypeError, (q, q, k, k, out, lse), dict(dq=q.half())),
        (ValueError, (q, q, k, k, out, lse), dict(dq=t(2, 5, 1, 64).expand(2, 5, 4, 64))),
    ]:
        with pytest.raises(err):
            b(*args, **opts)
    assert out.sum() == 0


@pytest.mark.slow
def test_caches_of_more_than_2_31_elements():
    """The last sequence of such a cache against the same keys in a tensor of their own (two
    ways to cut the keys: each within the other's bound), forward in every form, and backward."""
    import coo_spmm_sparse_gb300 as sn
    g = gen(17)
    n, room, heads, d = 4, 70001, 64, 128
    k, v = (torch.empty(n, room, heads, d, device="cuda", dtype=BF16) for _ in range(2))
    assert k.numel() > 2 ** 31
    for i in range(n):
        k[i].normal_(generator=g)
        v[i].normal_(generator=g)
    for q_tokens in (1, 40, 256):
        q = rnd(g, (n, q_tokens, heads, d), BF16)
        fill = ints(5, 70001, 1000, 69990)
        out, lse = sn.snack_attention_forward(q, k, v, k_lengths=fill)
        for i in (1, 3):
            m = int(fill[i])
            alone, log = sn.snack_attention_forward(q[i: i + 1], k[i: i + 1, :m].clone(), v[i: i + 1, :m].clone())
            # 70000 keys of one size: a result is about 1/260, a probability off by 2^-8 of itself
            assert float((out[i].double() - alone[0].double()).abs().max()) <= 2.0 ** -8 * float(alone.abs().max()) + 1e-4
            assert torch.allclose(lse[:, i], log[:, 0], atol=1e-4)
    rows = slice(69000, 69200)
    ks, vs = (t[:, rows].expand(n, 200, heads, d) for t in (k, v))
    q, dout = (rnd(g, (n, 200, heads, d), BF16) for _ in range(2))
    out, lse = sn.snack_attention_forward(q, ks, vs)
    got = sn.snack_attention_backward(dout, q, ks, vs, out, lse)
    want = sn.snack_attention_backward(dout, q, ks.contiguous(), vs.contiguous(), out, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_wait_has_run_out():
    import coo_spmm_sparse_gb300 as sn
    assert not sn.snack_attention_error() and not sn.snack_attention_error(torch.cuda.Stream())
