"""Attention where sequences, heads and tokens lie far apart: in length, in place, in magnitude."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_the_longest_cache(dtype):
    """One key for 2^31 - 4097 tokens by a stride of zero: every probability is the same, and the
    log of the sum is that of the number of keys (each lane counts its own exactly; 2^-20 for the logs)."""
    import coo_spmm_sparse_gb300 as sn
    n = 2 ** 31 - 4097
    q = torch.zeros(1, 1, 1, 8, device="cuda", dtype=dtype)
    k = torch.ones(1, 1, 1, 8, device="cuda", dtype=dtype).expand(1, n, 1, 8)
    v = torch.arange(8.0, device="cuda").to(dtype).view(1, 1, 1, 8).expand(1, n, 1, 8)
    for dropout in (0.0, 0.5):
        out, lse = sn.snack_attention_forward(q, k, v, dropout=dropout, seed=1)
        assert abs(float(lse) - math.log(n)) <= 2.0 ** -20 * math.log(n)
        # half of 2^31 draws: off by some 2^-16 of them
        assert torch.allclose(out.flatten().double(), v[0, 0, 0].double(), rtol=2.0 ** -7 if dtype != F32 else 2.0 ** -12)


# ---------------------------------------------------------------- sequences far apart in magnitude




def run(q, k, v, dout, **opts):
    import coo_spmm_sparse_gb300 as sn
    out, lse = sn.snack_attention_forward(q, k, v, **opts)
    return (out, lse, *sn.snack_attention_backward(dout, q, k, v, out, lse, **opts))


def same_but_for_powers(got, want, power):
    """got = want * 2^power, bit for bit; float16 results that are subnormal may round apart."""
    w = want.double() * 2.0 ** power
    if got.dtype == F16:
        assert bool(((got.double() - w).abs() <= 2.0 ** -24 * max(1.0, 2.0 ** power)).all())
    else:
        assert torch.equal(got.double(), w)


def layouts(d, n, length):
    """(shape of a side, options, slices of the sequences): dense, padded and ragged; the sizes that
    take the tiles, and those that do not."""
    ends = torch.tensor([0, *([length] * n)]).cumsum(0).to(torch.int32).cuda()
    fill = torch.tensor([length - 37 * i for i in range(n)], dtype=torch.int32).cuda()
    per = [(i, slice(0, length)) for i in range(n)]
    return [((n, length), {}, per), ((n, length), dict(q_lengths=fill, k_lengths=fill), per),
            ((n * length,), dict(q_offsets=ends, k_offsets=ends), [slice(i * length, (i + 1) * length) for i in range(n)])]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length,d", [(40, 64), (700, 64), (700, 65), (700, 128), (515, 100)])
@pytest.mark.parametrize("dropout", [0.0, 0.2])
def test_a_sequence_does_not_change_with_the_others_magnitudes(dtype, length, d, dropout):
    """Sequence n's q, k, v and dout times powers of two of its own: its results are those times
    powers of two, whatever the others are.  (Nothing of a call may be scaled by what another
    sequence holds; powers of two change no rounding.)"""
    far = 4 if dtype == F16 else 24
    for shape, opts, at in layouts(d, 3, length):
        g = gen(length + d)
        q, k, v, dout = (rnd(g, (*shape, h, d), dtype) for h in (6, 2, 2, 6))
        if dtype == F16:  # no input may become subnormal
            q, k, v, dout = (t + torch.copysign(torch.full_like(t, 2.0 ** -4), t) for t in (q, k, v, dout))
        opts = dict(opts, dropout=dropout, seed=7)
        want = run(q, k, v, dout, **opts)
        for powers in (((0, 0, 0), (far, -far, far // 2), (-far, 0, -far)), ((0, 0, far), (0, far, 0), (far, 0, 0))):
            x = [t.clone() for t in (q, k, v, dout)]
            for s, (a, b, c) in zip(at, powers):
                b = 0 if dtype == F16 else b  # (out is an input of the backward call: as above)
                for t, p in zip(x, (a, -a, b, c)):
                    t[s] *= 2.0 ** p
            got = run(*x, **opts)
            assert torch.equal(got[1], want[1])
            for s, (a, b, c) in zip(at, powers):
                b = 0 if dtype == F16 else b
                for y, w, p in zip((got[0], *got[2:]), (want[0], *want[2:]), (b, b + c - a, b + c + a, c)):
                    same_but_for_powers(y[s], w[s], p)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length,d", [(40, 64), (700, 64), (700, 65), (700, 128)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_what_is_not_finite_stays_in_its_sequence(dtype, length, d, value):
    for shape, opts, at in layouts(d, 3, length):
        g = gen(length + d)
        x = [rnd(g, (*shape, h, d), dtype) for h in (6, 2, 2, 6)]
        want = run(*x, **opts)
        for t in x:
            t[at[1]][20, 1, 3] = value
        got = run(*x, **opts)
        for s in (at[0], at[2]):
            for y, w in zip((got[0], *got[2:]), (want[0], *want[2:])):
                assert torch.equal(y[s], w[s])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ratio", [2.0 ** -7, 2.0 ** -13, 2.0 ** -17])
@pytest.mark.parametrize("length,d", [(1100, 64), (1100, 65), (1000, 128), (200, 64)])
def test_tokens_whose_gradients_lie_far_apart(dtype, ratio, length, d):
    """dq of a token is linear in its own dout, so that its bound is the bound of a call whose
    dout are all of one size, times its size.  Keys that only late tokens see have dk and dv
    bounded by what those tokens bring."""
    import attention_ref
    g = gen(d)
    q, k, v = (rnd(g, (1, length, h, d), dtype) for h in (4, 2, 2))
    dout = rnd(g, (1, length, 4, d), torch.float64, 256.0 if dtype == F16 else 1.0)
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # a step of a subnormal result
    every = torch.ones(length, device="cuda", dtype=torch.float64)
    every[1::2] = ratio
    late = torch.ones_like(every)
    late[length // 2:] = ratio
    for size in (every, late):
        size = size[None, :, None, None]
        x = (dout * size).to(dtype)
        flat = attention_ref.attention(q, k, v, dout=x.double() / size)
        _, _, dq, dk, dv = run(q, k, v, x)
        err = (dq.double() - flat["dq"][0] * size).abs()
        assert bool((err <= 1.01 * flat["dq"][1] * size + tiny).all()), float((err / (flat["dq"][1] * size)).max())
    first = (length // 2 + 127) // 128 * 128  # keys from here on: late tokens' only
    small = x.double() / ratio
    small[:, :length // 2] = 0
    want = attention_ref.attention(q, k, v, dout=small)
    for name, got in (("dk", dk), ("dv", dv)):
        ref, bound = (t[:, first:] * ratio for t in want[name])
        assert bool(((got[:, first:].double() - ref).abs() <= 1.01 * bound + tiny).all()), name


@pytest.mark.parametrize("length", [300, 1500])
def test_heads_whose_values_lie_far_apart(length):
    """32-bit operands are taken in parts scaled tile by tile and head by head: a head's results are
    those of the same head among others of its size."""
    g = gen(length)
    q, dout = (rnd(g, (2, length, 6, 64), F32) for _ in range(2))
    k, v = (rnd(g, (2, length, 3, 64), F32) for _ in range(2))
    want = run(q, k, v, dout)
    powers = torch.tensor([2.0 ** 30, 1.0, 2.0 ** -30], device="cuda")[:, None]
    both = powers.repeat_interleave(2, 0)
    got = run(q * both, k / powers, v * powers, dout * both.flip(0))
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0] * both)
    assert torch.equal(got[2], want[2] * both.flip(0)) and torch.equal(got[4], want[4] * powers.flip(0))
    assert torch.equal(got[3], want[3] * powers * powers * powers.flip(0))


# ---------------------------------------------------------------- queries that see few keys

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("form", ["wide", "long", "padded", "all", "ragged", "other", "odd"])
def test_queries_of_few_keys_do_not_read_out(dtype, form):
    """delta of a query that sees 2 to 32 keys comes from the tensors, whatever else is in the call:
    the gradients are the same, bit for bit, with another out in those rows.  The keys of the other
    queries do matter to it: with another out there dq changes."""
    import coo_spmm_sparse_gb300 as sn
    g = gen(21)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ends = lambda *v: ints(0, *torch.tensor(v).cumsum(0).tolist())  # noqa: E731
    heads, key_heads, d, causal, opts = 12, 4, 128, True, {}
    if form == "wide":  # many sequences of few tokens
        shape, kshape = (64, 33), (64, 33)
    elif form == "long":  # the first rows of long sequences
        shape = kshape = (2, 1500)
    elif form == "padded":
        shape = kshape = (5, 300)
        opts = dict(q_lengths=ints(300, 2, 20, 33, 0), k_lengths=ints(300, 2, 20, 33, 0))
    elif form == "all":  # every key seen
        shape, kshape, causal = (4, 200), (4, 600), False
        opts = dict(k_lengths=ints(32, 600, 5, 33))
    elif form == "ragged":
        at = ends(2, 0, 500, 31, 33, 1, 7)
        shape = kshape = (574,)
        opts = dict(q_offsets=at, k_offsets=at)
    elif form == "other":
        shape, kshape = (260,), (340,)
        opts = dict(q_offsets=ends(20, 200, 40), k_offsets=ends(22, 300, 18))
    else:
        shape, kshape, d = (3, 90), (3, 90), 65
    q, dout = (rnd(g, (*shape, heads, d), dtype) for _ in range(2))
    k, v = (rnd(g, (*kshape, key_heads, d), dtype) for _ in range(2))
    opts = dict(opts, causal=causal, dropout=0.2, seed=5)
    out, lse = sn.snack_attention_forward(q, k, v, **opts)
    want = sn.snack_attention_backward(dout, q, k, v, out, lse, **opts)
    few = torch.zeros(shape, dtype=torch.bool, device="cuda")
    if len(shape) == 1:
        qo, ko = opts["q_offsets"].tolist(), opts["k_offsets"].tolist()
        spans = [(slice(a, b), b - a, y - x) for a, b, x, y in zip(qo, qo[1:], ko, ko[1:])]
    else:
        ql = opts["q_lengths"].tolist() if "q_lengths" in opts else [shape[1]] * shape[0]
        kl = opts["k_lengths"].tolist() if "k_lengths" in opts else [kshape[1]] * shape[0]
        spans = [((n, slice(0, a)), a, b) for n, (a, b) in enumerate(zip(ql, kl))]
    for at, nq, nk in spans:
        i = torch.arange(nq, device="cuda")
        few[at] = (i + nk - nq + 1 if causal else i * 0 + nk) <= 32
    assert few.any() and not few.all()
    other = torch.where(few[..., None, None], out * (1 + torch.finfo(dtype).eps), out)
    got = sn.snack_attention_backward(dout, q, k, v, other, lse, **opts)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rest = torch.where(few[..., None, None], out, out * 1.5)
    assert not torch.equal(sn.snack_attention_backward(dout, q, k, v, rest, lse, **opts)[0], want[0])
    import attention_ref
    attention_ref.assert_within(dict(zip(("dq", "dk", "dv"), want)),
                                attention_ref.attention(q, k, v, dout=dout, **opts))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group,d", [(1, 64), (3, 128), (8, 80)])
def test_many_sequences_of_few_queries(dtype, group, d):
    """On both sides of the rules that go by the rows of a sequence: decoding large batches, packed
    requests of 1 to 20 new tokens, one long sequence among many short ones."""
    import attention_ref
    import coo_spmm_sparse_gb300 as sn
    g = gen(group)
    for n, nq, nk in ((200, 1, 100), (150, 32 // group, 70), (150, 32 // group + 1, 70)):
        q, k, v = (rnd(g, (n, t, h, d), dtype) for t, h in ((nq, 2 * group), (nk, 2), (nk, 2)))
        fill = torch.randint(nq, nk + 1, (n,), generator=g, device="cuda").to(torch.int32)
        opts = dict(k_lengths=fill, dropout=0.2, seed=1)
        got = sn.snack_attention_forward(q, k, v, **opts)
        attention_ref.assert_within(dict(zip(("out", "lse"), got)), attention_ref.attention(q, k, v, **opts))
    for lq, lk in (([1] * 128, [90] * 128), ([15] * 150, [20] * 150), ([16] * 150, [16] * 150),
                   ([1500] + [1] * 100, [1500] + [3] * 100), ([0, 20, 1] * 40, [5, 40, 0] * 40)):
        ends = [torch.tensor([0, *l], device="cuda").cumsum(0).to(torch.int32) for l in (lq, lk)]
        q, k, v = (rnd(g, (t, h, d), dtype) for t, h in ((sum(lq), 2 * group), (sum(lk), 2), (sum(lk), 2)))
        opts = dict(q_offsets=ends[0], k_offsets=ends[1])
        got = sn.snack_attention_forward(q, k, v, **opts)
        attention_ref.assert_within(dict(zip(("out", "lse"), got)), attention_ref.attention(q, k, v, **opts))


# ---------------------------------------------------------------- waits that give up

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length", [300, 1024])
def test_waits_that_give_up_leave_nan_and_the_flag(dtype, d, length):
    """Every wait of the tiles gives up at once: all results are NaN, the flag is set and is cleared by
    reading it, and the calls that follow are right.  (32 bits at 128 columns: no tiles, no waits.)"""
    import coo_spmm_sparse_gb300 as sn
    g = gen(22)
    q, k, v, dout = (rnd(g, (8, length, h, d), dtype) for h in (8, 4, 4, 8))
    want = run(q, k, v, dout)
    torch.cuda.synchronize()
    assert not sn.snack_attention_error()
    try:
        sn.snack_debug_attention_polls(0)
        out, lse = sn.snack_attention_forward(q, k, v)
        grads = sn.snack_attention_backward(dout, q, k, v, want[0], want[1])
        torch.cuda.synchronize()
        tiles = dtype != F32 or d == 64
        assert sn.snack_attention_error() == tiles and not sn.snack_attention_error()
        for t in (out, lse, *grads) if tiles else ():
            assert t.isnan().all()
    finally:
        sn.snack_debug_attention_polls(-1)
    assert all(torch.equal(a, b) for a, b in zip(run(q, k, v, dout), want))
    assert not sn.snack_attention_error()


def test_waits_that_give_up_with_keys_in_parts():
    import coo_spmm_sparse_gb300 as sn
    g = gen(23)
    q, k, v = (rnd(g, (1, n, 8, 64), BF16) for n in (130, 9000, 9000))
    want = sn.snack_attention_forward(q, k, v)
    try:
        sn.snack_debug_attention_polls(0)
        out, lse = sn.snack_attention_forward(q, k, v)
        assert sn.snack_attention_error() and out.isnan().all() and lse.isnan().all()
    finally:
        sn.snack_debug_attention_polls(-1)
    assert all(torch.equal(a, b) for a, b in zip(sn.snack_attention_forward(q, k, v), want))


# ---------------------------------------------------------------- how far off 16-bit gradients are

@pytest.mark.parametrize("n,length,heads,key_heads,d", [(2, 1024, 8, 4, 64), (1, 2048, 8, 2, 128), (4, 300, 12, 12, 64)])
def test_bfloat16_gradients_are_as_exact_as_their_rounding(n, length, heads, key_heads, d):
    """Probabilities and gradients of scores in two parts leave dq, dk and dv where rounding them to
    bfloat16 alone does: with errors that add up like independent ones, delta of a rounded out
    (2^-9 of a sum that cancels to about 2 of its size) may add a tenth; one part of either adds half."""
    import attention_ref
    g = gen(24)
    q, k, v, dout = (rnd(g, (n, length, h, d), BF16) for h in (heads, key_heads, key_heads, heads))
    got = run(q, k, v, dout)
    want = attention_ref.attention(q, k, v, dout=dout)
    for name, t in zip(("dq", "dk", "dv"), got[2:]):
        ref = want[name][0]
        off, least = ((x.double() - ref).norm() for x in (t, ref.to(BF16)))
        assert float(off) <= 1.1 * float(least), (name, float(off / least))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("side", ["keys", "queries"])
def test_gradients_of_scores_that_grow_along_a_row(dtype, d, side):
    """Values, or dout, 16 times as large every 128 tokens: a row's power falls from step to step, and
    sums that stay in tensor memory are multiplied down with it."""
    import attention_ref
    g = gen(25)
    n = 640
    q, k, v, dout = (rnd(g, (2, n, h, d), torch.float64) for h in (4, 2, 2, 4))
    growth = (16.0 ** (torch.arange(n, device="cuda") // 128) / 256.0)[None, :, None, None]
    if side == "keys":
        v = v * growth
    else:
        dout = dout * growth
    q, k, v, dout = (t.to(dtype) for t in (q, k, v, dout))
    for causal in (True, False):
        got = run(q, k, v, dout, causal=causal)
        want = attention_ref.attention(q, k, v, dout=dout, causal=causal)
        attention_ref.assert_within(dict(zip(("out", "lse", "dq", "dk", "dv"), got)), want)
        # and by the norm of each block of 128 tokens, which the largest does not cover
        u = {F32: 2.0 ** -16, BF16: 2.0 ** -7, F16: 2.0 ** -9}[dtype]
        for name, t in zip(("dq", "dk", "dv"), got[2:]):
            for at in range(0, n, 128):
                ref = want[name][0][:, at: at + 128]
                assert float((t[:, at: at + 128].double() - ref).norm()) <= u * float(ref.norm()), (name, at)


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("d", [72, 128])
def test_long_bfloat16_sequences_do_not_change_with_the_others(ragged, d):
    """The sizes whose operands are made in float16: powers of two and what is not finite, as above."""
    n, length = 3, 4200
    shape, opts, at = layouts(d, n, length)[2 if ragged else 0]
    g = gen(d)
    x = [rnd(g, (*shape, h, d), BF16) for h in (12, 4, 4, 12)]
    opts = dict(opts, dropout=0.1, seed=3)
    want = run(*x, **opts)
    powers = ((0, 0, 0), (24, -24, 12), (-24, 0, -24))
    y = [t.clone() for t in x]
    for s, (a, b, c) in zip(at, powers):
        for t, p in zip(y, (a, -a, b, c)):
            t[s] *= 2.0 ** p
    got = run(*y, **opts)
    assert torch.equal(got[1], want[1])
    for s, (a, b, c) in zip(at, powers):
        for u, w, p in zip((got[0], *got[2:]), (want[0], *want[2:]), (b, b + c - a, b + c + a, c)):
            same_but_for_powers(u[s], w[s], p)
    for t in x:
        t[at[1]][20, 1, 3] = math.nan
    got = run(*x, **opts)
    for s in (at[0], at[2]):
        for u, w in zip((got[0], *got[2:]), (want[0], *want[2:])):
            assert torch.equal(u[s], w[s])


@pytest.mark.parametrize("d,causal,dropout", [(128, True, 0.0), (80, False, 0.0), (128, True, 0.2), (65, True, 0.0)])
def test_long_bfloat16_gradients(d, causal, dropout):
    """Against 64 bits, and, as long sequences' bounds are wide, as exact as their rounding (a tenth
    for delta of the rounded out); then with dout of every other token 2^-17 of the rest."""
    import attention_ref
    g = gen(d)
    n, heads = 7200, 12
    q, k, v, dout = (rnd(g, (1, n, h, d), BF16) for h in (heads, 4, 4, heads))
    opts = dict(causal=causal, dropout=dropout, seed=2)
    size = torch.ones(n, device="cuda", dtype=torch.float64)
    size[1::2] = 2.0 ** -17
    size = size[None, :, None, None]
    for scale in (torch.ones_like(size), size):
        x = (dout.double() * scale).to(BF16)
        got = run(q, k, v, x, **opts)
        for h in range(4):  # a key head at a time: the reference holds its probabilities
            at = slice(3 * h, 3 * h + 3)
            if dropout:  # (the mask goes by all heads; the heads' own reference needs it all)
                break
            want = attention_ref.attention(q[:, :, at], k[:, :, h: h + 1], v[:, :, h: h + 1], dout=x[:, :, at], causal=causal)
            attention_ref.assert_within({"out": got[0][:, :, at], "dv": got[4][:, :, h: h + 1],
                                         "dk": got[3][:, :, h: h + 1], "dq": got[2][:, :, at]}, want)
            ref = want["dq"][0] / scale
            off, least = (((t.double() / scale) - ref).norm() for t in (got[2][:, :, at], want["dq"][0].to(BF16)))
            assert float(off) <= 1.1 * float(least), float(off / least)
            for name, t in (("dk", got[3]), ("dv", got[4])):
                ref = want[name][0]
                off, least = ((y.double() - ref).norm() for y in (t[:, :, h: h + 1], ref.to(BF16)))
                assert float(off) <= 1.1 * float(least), (name, float(off / least))
            del want
    if dropout:  # dv by its linearity in dout: a single row's
        x = torch.zeros_like(dout)
        x[:, 5000] = dout[:, 5000]
        out, lse, _, _, dv = run(q, k, v, x, **opts)
        M = attention_ref.mask_of(2, (torch.tensor([5000 * heads], device="cuda") + torch.arange(heads, device="cuda")) << 30,
                                  n, dropout)
        s = torch.einsum("hd,jhd->hj", q[0, 5000].double(), k[0].double().repeat_interleave(3, 1)) * d ** -0.5
        P = torch.softmax(s[:, :5001], -1) * M[:, :5001]
        want = torch.einsum("hj,hd->jhd", P, dout[0, 5000].double()).view(5001, 4, 3, d).sum(2)
        terms = torch.einsum("hj,hd->jhd", P, dout[0, 5000].double().abs()).view(5001, 4, 3, d).sum(2)
        assert bool(((dv[0, :5001].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 2.0 ** -9 * terms + 1e-12).all())
        assert not dv[0, 5001:].any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("form", ["offset", "repeated", "odd strides"])
def test_a_gradient_that_lies_badly_takes_the_same_path(dtype, form):
    """The same bits as from a copy of it (mma.sync would differ in some)."""
    import coo_spmm_sparse_gb300 as sn
    g = gen(26)
    q, k, v = (rnd(g, (2, 500, h, 64), dtype) for h in (8, 4, 4))
    if form == "offset":
        dout = rnd(g, (2 * 500 * 8 * 64 + 4,), dtype)[4:].view(2, 500, 8, 64)
    elif form == "repeated":
        dout = rnd(g, (2, 500, 1, 64), dtype).expand(2, 500, 8, 64)
    else:
        dout = rnd(g, (2, 500, 8, 65), dtype)[..., :64]
    out, lse = sn.snack_attention_forward(q, k, v)
    got = sn.snack_attention_backward(dout, q, k, v, out, lse)
    want = sn.snack_attention_backward(dout.contiguous().clone(), q, k, v, out, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,length,d", [(F32, 700, 64), (F32, 515, 40), (F16, 700, 128), (BF16, 700, 64),
                                            (BF16, 4200, 128)])
def test_dense_and_ragged_sides_in_any_mix(dtype, length, d):
    """The same sequences dense, padded or packed on either side: the same bits (tiles, and the powers
    of two of their operands, are found by unlike numberings)."""
    g = gen(27)
    n, heads, key_heads = 3, 12, 4
    q, k, v, dout = (rnd(g, (n, length, h, d), dtype) for h in (heads, key_heads, key_heads, heads))
    q[1] *= 16.0
    v[2] *= 2.0 ** -10 if dtype != F16 else 0.25
    ends = (torch.arange(n + 1, device="cuda") * length).to(torch.int32)
    full = torch.full((n,), length, dtype=torch.int32, device="cuda")
    opts = dict(dropout=0.1, seed=4)
    want = run(q, k, v, dout, **opts)
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    for q_form in ("dense", "padded", "ragged"):
        for k_form in ("dense", "padded", "ragged"):
            o = dict(opts)
            x = [flat(t) if form == "ragged" else t for t, form in zip((q, k, v, dout), (q_form, k_form, k_form, q_form))]
            for side, form in (("q", q_form), ("k", k_form)):
                if form != "dense":
                    o[f"{side}_offsets" if form == "ragged" else f"{side}_lengths"] = ends if form == "ragged" else full
            got = run(*x, **o)
            for a, b in zip(got, want):
                assert torch.equal(a.reshape(-1), b.reshape(-1)), (q_form, k_form)


@pytest.mark.parametrize("dtype,length,d", [(F32, 700, 64), (F16, 700, 64), (BF16, 700, 128), (BF16, 7300, 128)])
def test_replays_take_their_powers_from_their_own_inputs(dtype, length, d):
    """A captured call whose inputs are replaced by ones 2^12 times smaller, and back: each replay's
    results are those of an eager call on the same inputs (no largest magnitude stays behind)."""
    g = gen(28)
    x = [rnd(g, (1, length, h, d), dtype) for h in (12, 4, 4, 12)]
    room = [t.clone() for t in x]
    run(*room)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(*room)
    by = 2.0 ** -12 if dtype != F16 else 2.0 ** -3
    for scale in (1.0, by, 1.0):
        for r, t in zip(room, x):
            r.copy_(t * scale)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, run(*room)))
