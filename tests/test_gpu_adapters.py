"""Adapters of many requests beside a projection, against a 64-bit evaluation
request by request (bounds in dense_ref.py), their gradients also against
differences, and what the calls refuse."""

import pytest
import torch

import dense_ref
from dense_ref import assert_within

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def make(offsets, which, N, inp, out, rank, dt, T=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = offsets[-1] if T is None else T

    def rnd(s, std=1.0):
        return (torch.randn(s, generator=g, device="cuda") * std).to(dt)

    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(X=rnd((T, inp)), Y=rnd((T, out)), A=rnd((N, rank, inp), inp ** -0.5),
                B=rnd((N, out, rank), rank ** -0.5), offsets=torch.tensor(offsets, **i32),
                which=torch.tensor(which, **i32),
                scale=torch.rand(N, generator=g, device="cuda") + 0.5,
                dY=rnd((T, out)), dX=rnd((T, inp)))


def check(c, train=True, have_dx=True):
    import coo_spmm_sparse_gb300 as sn
    args = (c["A"], c["B"], c["offsets"], c["which"], c["scale"])
    want = dense_ref.adapter(c["X"], c["Y"], *args, dY=c["dY"] if train else None,
                             dX=c["dX"] if have_dx else None)
    Y, H = sn.snack_adapter_forward(c["X"], *args, c["Y"])
    assert Y is c["Y"]
    got = {"Y": Y, "H": H}
    if train:
        got["dX"], got["dA"], got["dB"] = sn.snack_adapter_backward(
            c["X"], c["dY"], *args, H, dX=c["dX"] if have_dx else None)
    torch.cuda.synchronize()
    for k, v in got.items():
        assert_within(k, v, *want[k])
    return got


RAGGED = ([0, 3, 3, 20, 21, 85, 90, 217], [2, 0, 1, 2, -1, 0, 1])


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("rank", [1, 2, 4, 5, 8, 12, 16, 17, 32, 33, 64, 72, 130])
def test_every_rank(dt, rank):
    check(make(*RAGGED, 4, 192, 320, rank, dt, seed=rank))


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("inp,out", [(1, 1), (3, 5), (33, 7), (64, 64), (100, 1001), (255, 130),
                                     (768, 2304), (1000, 96), (2304, 40)])
def test_every_width(dt, inp, out):
    check(make(*RAGGED, 3, inp, out, 8, dt, seed=inp))
    check(make(*RAGGED, 3, inp, out, 20, dt, seed=inp + 1))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 15, 16, 17, 64, 65, 128, 200])
def test_one_token_per_request(dt, T):
    g = torch.Generator().manual_seed(T)
    which = torch.randint(-1, 7, (T,), generator=g).tolist()
    check(make(list(range(T + 1)), which, 7, 160, 96, 16, dt, seed=T))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [64, 65, 96, 97, 300])
@pytest.mark.parametrize("inp,out,rank", [(2304, 768, 12), (1001, 4096, 33), (64, 2048, 16)])
def test_few_tiles_of_wide_rows(dt, T, inp, out, rank):
    check(make([0, 7, 50, T], [1, 0, 1], 2, inp, out, rank, dt, seed=T))


@pytest.mark.parametrize("T,R,N", [(1, 1, 1), (700, 1, 1), (1500, 40, 3), (1031, 9, 30),
                                   (300, 300, 2), (2100, 1500, 40)])
def test_many_requests_and_tokens(T, R, N):
    g = torch.Generator().manual_seed(T + R)
    cut = torch.randint(0, T + 1, (R - 1,), generator=g).sort().values.tolist()
    which = torch.randint(-1, N, (R,), generator=g).tolist()
    check(make([0] + cut + [T], which, N, 128, 144, 8, F32, seed=T))
    check(make([0] + cut + [T], which, N, 128, 144, 24, BF16, seed=T))


def test_tokens_outside_requests_and_adapters_out_of_range():
    c = make([5, 9, 40, 60], [1, 9, 0], 2, 96, 64, 8, F32, T=77)
    y0, dx0 = c["Y"].clone(), c["dX"].clone()
    got = check(c)
    for rows in (slice(0, 5), slice(9, 40), slice(60, 77)):
        assert torch.equal(got["Y"][rows], y0[rows])
        assert torch.equal(got["dX"][rows], dx0[rows])
        assert not got["H"][rows].any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_no_adapter_is_used(dt):
    c = make([0, 10, 30], [-1, -1], 3, 64, 64, 16, dt)
    y0 = c["Y"].clone()
    got = check(c)
    assert torch.equal(got["Y"], y0) and not got["dA"].any() and not got["dB"].any()


def test_nothing():
    import coo_spmm_sparse_gb300 as sn
    c = make([0, 0], [0], 2, 32, 48, 4, F32)
    assert c["X"].shape[0] == 0
    got = check(c)
    assert not got["dA"].any() and not got["dB"].any()
    c = make([0], [], 2, 32, 48, 4, F32, T=6)
    check(c)
    Y, H = sn.snack_adapter_forward(c["X"], c["A"][:0], c["B"][:0], c["offsets"], c["which"], 1.0,
                                    c["Y"])
    assert H.shape == (6, 4)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("pad,at", [(8, 0), (16, 8), (5, 0), (7, 3)])
def test_strided_rows_and_misaligned_starts(dt, pad, at):
    c = make(*RAGGED, 3, 96, 128, 16, dt, seed=pad)

    def wide(t):
        v = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=dt, device="cuda")[:, at: at + t.shape[1]]
        v.copy_(t)
        return v

    for k in ("X", "Y", "dX", "dY"):
        c[k] = wide(c[k])
    check(c)


@pytest.mark.parametrize("T", [40, 200])
@pytest.mark.parametrize("size", [2.0 ** -14, 1.0, 2.0 ** 9])
def test_float16_beyond_its_range(T, size):
    """H of up to 2^18 and gradients of 2^-14 in float16: what lies between the
    two products never is a float16."""
    c = make([0, 9, T], [1, 0], 2, 192, 160, 16, F16, seed=T)
    c["X"] = (c["X"].float() * size).half()
    c["A"] = (c["A"].float() * max(1.0, size / 8)).half()
    c["B"] = (c["B"].float() / max(1.0, size * size / 8)).half()
    c["dY"] = (c["dY"].float() * min(size, 1 / size)).half()
    check(c)


def test_values_of_the_rest_do_not_leak():
    """NaN in tokens without an adapter, and in adapters that no request names, reach nothing else."""
    import coo_spmm_sparse_gb300 as sn
    for dt in (F32, BF16):
        c = make([0, 40, 41, 90], [1, -1, 0], 4, 128, 96, 16, dt, seed=2)
        want = dense_ref.adapter(c["X"], c["Y"], c["A"], c["B"], c["offsets"], c["which"],
                                 c["scale"], dY=c["dY"], dX=c["dX"])
        nan = float("nan")
        c["X"][40], c["dY"][40] = nan, nan
        c["A"][2:], c["B"][2:], c["scale"][2:] = nan, nan, nan
        args = (c["A"], c["B"], c["offsets"], c["which"], c["scale"])
        Y, H = sn.snack_adapter_forward(c["X"], *args, c["Y"])
        dX, dA, dB = sn.snack_adapter_backward(c["X"], c["dY"], *args, H, dX=c["dX"])
        for k, v in (("Y", Y), ("dX", dX), ("dA", dA), ("dB", dB)):
            assert_within(k, v, *want[k])


def test_uniform_scale_parts_and_fresh_dx():
    import coo_spmm_sparse_gb300 as sn
    c = make(*RAGGED, 3, 128, 64, 8, F32, seed=3)
    c["scale"] = 0.25
    check(c, have_dx=False)
    args = (c["A"], c["B"], c["offsets"], c["which"], c["scale"])
    _, H = sn.snack_adapter_forward(c["X"], *args, c["Y"].clone())
    dX, dA, dB = sn.snack_adapter_backward(c["X"], c["dY"], *args, H)
    a, b, _ = sn.snack_adapter_backward(c["X"], c["dY"], *args, H, need_dw=False)
    assert b is None and torch.equal(a, dX)
    a, b, d = sn.snack_adapter_backward(c["X"], c["dY"], *args, H, need_dx=False)
    assert a is None and torch.equal(b, dA) and torch.equal(d, dB)


def test_gradients_against_differences():
    """The loss sum(Y c) is linear in X, A and B each: a central difference of
    any step is the derivative up to rounding (2^-24 of ~7000 terms of order
    1); held to 1e-4 of the terms' 2-norm and 0.1."""
    import coo_spmm_sparse_gb300 as sn
    c = make([0, 6, 11, 24], [1, 0, 1], 2, 80, 72, 8, F32, seed=4)
    args = [c["A"], c["B"], c["offsets"], c["which"], c["scale"]]
    zero = torch.zeros_like(c["Y"])
    _, H = sn.snack_adapter_forward(c["X"], *args, zero.clone())
    dX, dA, dB = sn.snack_adapter_backward(c["X"], c["dY"], *args, H)
    g = torch.Generator(device="cuda").manual_seed(8)
    for base, grad, put in ((c["X"], dX, "X"), (c["A"], dA, 0), (c["B"], dB, 1)):
        e = torch.randn(base.shape, generator=g, device="cuda")
        loss = []
        for step in (0.5, -0.5):
            v, a = base + step * e, list(args)
            if put == "X":
                y, _ = sn.snack_adapter_forward(v, *a, zero.clone())
            else:
                a[put] = v
                y, _ = sn.snack_adapter_forward(c["X"], *a, zero.clone())
            loss.append((y.double() * c["dY"].double()).sum())
        terms = grad.double() * e.double()
        assert abs(float(terms.sum()) - float(loss[0] - loss[1])) <= 1e-4 * float(terms.norm()) + 0.1


def test_same_bits_every_time_and_on_another_stream():
    import coo_spmm_sparse_gb300 as sn
    for dt, r in ((F32, 16), (BF16, 8)):
        c = make([0, 300, 301, 900, 1500], [0, 1, 1, 0], 2, 512, 640, r, dt, seed=6)
        args = (c["A"], c["B"], c["offsets"], c["which"], c["scale"])

        def once():
            Y, H = sn.snack_adapter_forward(c["X"], *args, c["Y"].clone())
            return (Y, H) + sn.snack_adapter_backward(c["X"], c["dY"], *args, H,
                                                      dX=c["dX"].clone())

        first = once()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = once()
        torch.cuda.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [40, 300])
def test_fresh_dx_on_a_given_stream(T):
    """What the call allocates and clears is in the order of the stream it is
    given, not of the current one, which is kept busy here."""
    import coo_spmm_sparse_gb300 as sn
    c = make([0, 9, T], [1, 0], 2, 256, 192, 8, F32, seed=7)
    args = (c["A"], c["B"], c["offsets"], c["which"], c["scale"])
    want = dense_ref.adapter(c["X"], c["Y"], *args, dY=c["dY"])
    busy = torch.randn(8192, 8192, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        busy = busy @ busy * 1e-4
    Y, H = sn.snack_adapter_forward(c["X"], *args, c["Y"], stream=s)
    dX, dA, dB = sn.snack_adapter_backward(c["X"], c["dY"], *args, H, stream=s)
    torch.cuda.synchronize()
    for k, v in (("Y", Y), ("H", H), ("dX", dX), ("dA", dA), ("dB", dB)):
        assert_within(k, v, *want[k])


def test_module_beside_a_sparse_layer():
    import coo_spmm_sparse_gb300 as sn
    lin = sn.SnackLinear(256, 192, 5000, seed=1)
    lin.weight_values.requires_grad_(False)
    ad = sn.SnackAdapters(3, 256, 192, 8, alpha=16.0, seed=2)
    x = torch.randn(40, 256, device="cuda", requires_grad=True)
    off = torch.tensor([0, 10, 11, 40], dtype=torch.int32, device="cuda")
    which = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    base = lin(x).detach()
    assert torch.equal(ad(x, lin(x), off, which).detach(), base)  # B is zero: nothing changes
    with torch.no_grad():
        ad.B.normal_(0, 0.3)
    y = ad(x, lin(x), off, which)
    y.square().sum().backward()
    x64 = x.detach().double().requires_grad_()
    A, B = (p.detach().double().requires_grad_() for p in (ad.A, ad.B))
    row, col, val = lin.export()
    W = torch.zeros(192, 256, dtype=torch.float64, device="cuda")
    W[torch.from_numpy(row).long().cuda(), torch.from_numpy(col).long().cuda()] = \
        torch.from_numpy(val).double().cuda()
    parts = [x64[:10] @ A[2].T @ B[2].T * 2, x64[10:11] @ W.T * 0, x64[11:] @ A[0].T @ B[0].T * 2]
    y64 = x64 @ W.T + torch.cat(parts)
    y64.square().sum().backward()
    for got, want in ((y, y64), (x.grad, x64.grad), (ad.A.grad, A.grad), (ad.B.grad, B.grad)):
        assert torch.allclose(got.double(), want, rtol=1e-4, atol=1e-5 * float(want.abs().max()))


def test_refusals():
    import coo_spmm_sparse_gb300 as sn
    c = make([0, 4], [0], 2, 32, 48, 4, F32)
    f = sn.snack_adapter_forward
    ok = [c["X"], c["A"], c["B"], c["offsets"], c["which"], c["scale"], c["Y"]]

    def swap(i, v):
        a = list(ok)
        a[i] = v
        return a

    for i, v in ((0, c["X"].cpu()), (0, c["X"].double()), (1, c["A"].bfloat16()),
                 (3, c["offsets"].long()), (4, c["which"].cpu()), (6, c["Y"].bfloat16())):
        with pytest.raises(TypeError):
            f(*swap(i, v))
    for i, v in ((0, c["X"][:, :8]), (2, c["B"][..., :3]), (2, c["B"].transpose(1, 2)),
                 (3, c["offsets"][:1]), (5, c["scale"][:1]), (6, c["Y"][:3]),
                 (6, c["Y"][:, :8]), (0, c["X"].t())):
        with pytest.raises(ValueError):
            f(*swap(i, v))
    with pytest.raises(ValueError):
        f(*ok, H=torch.zeros(4, 5, device="cuda"))
    sq = make([0, 4], [0], 2, 32, 32, 4, F32)
    with pytest.raises(sn.SnackError) as e:
        f(sq["X"], sq["A"], sq["B"], sq["offsets"], sq["which"], 1.0, sq["X"])
    assert e.value.status == 1 and "overlaps" in str(e.value)
    big = make([0, 4], [0], 1, 8, 8, 513, F32)
    with pytest.raises(sn.SnackError) as e:
        f(big["X"], big["A"], big["B"], big["offsets"], big["which"], 1.0, big["Y"])
    assert e.value.status == 1 and "rank" in str(e.value)
    _, H = f(*ok)
    with pytest.raises(ValueError):
        sn.snack_adapter_backward(c["X"], c["dY"], *ok[1:6], H[:2])
    with pytest.raises(sn.SnackError) as e:
        sn.snack_adapter_backward(sq["X"], sq["dY"], sq["A"], sq["B"], sq["offsets"], sq["which"],
                                  1.0, H, dX=sq["dY"])
    assert e.value.status == 1


def test_second_derivatives_raise():
    """The backward's results carry no graph: differentiating them again
    raises, whatever the incoming gradient, where a constant would be wrong."""
    import coo_spmm_sparse_gb300 as sn
    ad = sn.SnackAdapters(2, 64, 48, 4, seed=3)
    with torch.no_grad():
        ad.B.normal_(0, 0.3)
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    which = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    for loss in (lambda y: y.sum(), lambda y: y.square().sum()):
        x = torch.randn(9, 64, device="cuda", requires_grad=True)
        for t in (x, ad.A, ad.B):
            y = ad(x, torch.zeros(9, 48, device="cuda"), off, which)
            g, = torch.autograd.grad(loss(y), t, create_graph=True)
            with pytest.raises(RuntimeError, match="second derivative"):
                (y.sum() + g.square().sum()).backward()


def test_a_scale_that_wants_a_gradient_is_refused():
    import coo_spmm_sparse_gb300 as sn
    ad = sn.SnackAdapters(2, 64, 48, 4, seed=3)
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    which = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    x = torch.randn(9, 64, device="cuda", requires_grad=True)
    ad.scale = torch.ones(2, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="scale"):
        ad(x, torch.zeros(9, 48, device="cuda"), off, which)
    ad.scale = torch.ones(2, device="cuda")
    ad(x, torch.zeros(9, 48, device="cuda"), off, which).sum().backward()


def test_writes_in_place_are_seen_by_autograd():
    """A tensor that autograd keeps for a backward pass and a call then
    changes: the backward pass raises, it does not use the changed values."""
    import coo_spmm_sparse_gb300 as sn
    c = make([0, 9, 40], [1, 0], 2, 64, 48, 8, F32, seed=9)
    args = (c["A"], c["B"], c["offsets"], c["which"], c["scale"])
    w = torch.ones(48, device="cuda", requires_grad=True)
    z = (c["Y"] * w).sum()
    _, H = sn.snack_adapter_forward(c["X"], *args, c["Y"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    w = torch.ones(64, device="cuda", requires_grad=True)
    z = (c["dX"] * w).sum()
    sn.snack_adapter_backward(c["X"], c["dY"], *args, H, dX=c["dX"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    w = torch.ones(8, device="cuda", requires_grad=True)
    z = (H * w).sum()
    sn.snack_adapter_forward(c["X"], *args, c["Y"], H=H)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    with torch.inference_mode():  # tensors without a version
        c = make([0, 9, 40], [1, 0], 2, 64, 48, 8, F32, seed=9)
        check(c)


@pytest.mark.parametrize("which", [[0, 1], [1, 0]])
def test_float16_adapters_of_unlike_magnitudes(which):
    """Two adapters whose H and dH lie 2^36 apart, side by side in one call:
    each one's gradients are those that it has alone."""
    c = make([0, 70, 150], which, 2, 192, 160, 8, F16, seed=10)
    small = slice(0, 70) if which[0] == 1 else slice(70, 150)
    large = slice(70, 150) if which[0] == 1 else slice(0, 70)
    for k, f in (("X", 2.0 ** -12), ("dY", 2.0 ** 9)):  # adapter 1: H of 2^-24, dB of 2^-12
        c[k][small] = (c[k][small].float() * f).half()
    c["A"][1] = (c["A"][1].float() * 2.0 ** -9).half()
    c["B"][1] = (c["B"][1].float() * 2.0 ** -9).half()
    for k, f in (("X", 2.0 ** 9), ("dY", 2.0 ** -9)):   # adapter 0: H of 2^12
        c[k][large] = (c[k][large].float() * f).half()
    c["A"][0] = (c["A"][0].float() * 2.0 ** 3).half()
    c["B"][0] = (c["B"][0].float() * 2.0 ** -6).half()
    check(c)


@pytest.mark.parametrize("rank", [64, 512])
def test_sums_over_high_ranks(rank):
    """Terms of one sign, where a sum that is cut off rather than rounded at
    every step drifts: H exact (one-hot rows of X pick weights of 8 bits), all
    of B positive.  Held to 3e-6 of the sum: 2^-21 for the split of a product,
    2^-24 on average for each of the 24 steps of 64 summed elements in the
    matrix unit, cut off between 0 and 2^-23 (1.4e-6, and 7e-7 for the spread of
    24 such cuts over the outputs), 2^-25 for each of 8 sums outside it."""
    import coo_spmm_sparse_gb300 as sn
    T, inp, out = 200, 64, 192
    c = make([0, T], [0], 1, inp, out, rank, F32, seed=rank)
    g = torch.Generator(device="cuda").manual_seed(1)
    c["X"] = torch.zeros(T, inp, device="cuda")
    c["X"][torch.arange(T), torch.arange(T) % inp] = 1.0
    c["A"] = torch.randint(128, 256, c["A"].shape, generator=g, device="cuda").float()
    c["B"] = torch.rand(c["B"].shape, generator=g, device="cuda") + 0.5
    Y, H = sn.snack_adapter_forward(c["X"], c["A"], c["B"], c["offsets"], c["which"], 1.0,
                                    torch.zeros(T, out, device="cuda"))
    assert torch.equal(H, c["X"] @ c["A"][0].T)
    want = H.double() @ c["B"][0].double().T
    worst = ((Y.double() - want).abs() / want).max()
    print("worst", rank, float(worst))
    assert float(worst) <= 3e-6


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("rank", [131, 256, 300, 512])
@pytest.mark.parametrize("T", [60, 150])
def test_high_ranks(dt, rank, T):
    check(make([0, 33, 90 if T > 90 else 40, T], [1, 0, 1], 2, 96, 160, rank, dt, T=T, seed=rank))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [40, 200])
def test_column_ranges_of_one_buffer(dt, T):
    """X and Y, and X, dY and dX, side by side in the rows of one buffer:
    ranges that share no element are no overlap."""
    import coo_spmm_sparse_gb300 as sn
    c = make([0, 9, T], [1, 0], 2, 96, 128, 8, dt, seed=T)
    wide = torch.zeros(T, 96 + 128 + 128 + 96, dtype=dt, device="cuda")
    at = 0
    for k in ("X", "Y", "dY", "dX"):
        v = wide[:, at: at + c[k].shape[1]]
        v.copy_(c[k])
        at += c[k].shape[1]
        c[k] = v
    check(c)
    args = (c["A"], c["B"], c["offsets"], c["which"], c["scale"])
    for lo in (88, 95):  # Y's first columns are X's last
        with pytest.raises(sn.SnackError) as e:
            sn.snack_adapter_forward(c["X"], *args, wide[:, lo: lo + 128])
        assert e.value.status == 1 and "overlaps" in str(e.value)
    other = wide.view(-1)[: T * 224].view(T, 224)[:, 96:]  # rows of another length over the same memory
    with pytest.raises(sn.SnackError):
        sn.snack_adapter_forward(c["X"], *args, other)


@pytest.mark.parametrize("T", [40, 90, 200])
def test_offsets_out_of_order_stay_in_bounds(T):
    """Offsets that decrease or lie outside [0, tokens]: which request a token
    then belongs to is not defined; nothing outside the tensors is written,
    and every row is one of the three that its adapters can give."""
    import coo_spmm_sparse_gb300 as sn
    c = make([0, 30, 10, T + 50, -7, T - 3], [1, 0, 1, 0, 1], 2, 64, 96, 8, F32, T=T, seed=T)
    flat = torch.full(((T + 2) * 96,), 7.0, device="cuda")
    y0, Y = c["Y"].clone(), flat[96: 96 + T * 96].view(T, 96)
    Y.copy_(c["Y"])
    sn.snack_adapter_forward(c["X"], c["A"], c["B"], c["offsets"], c["which"], c["scale"], Y)
    assert (flat[:96] == 7).all() and (flat[-96:] == 7).all()
    rows = [y0] + [y0 + c["scale"][n] * (c["X"].double() @ c["A"][n].double().T
                                         @ c["B"][n].double().T) for n in range(2)]
    near = torch.stack([torch.isclose(Y.double(), v.double(), rtol=1e-4, atol=1e-4).all(1)
                        for v in rows])
    assert near.any(0).all()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in X, Y and dX: the last rows are as they are alone."""
    import coo_spmm_sparse_gb300 as sn
    T, inp, rank = 530_000, 4096, 8
    g = torch.Generator(device="cuda").manual_seed(11)
    X, Y, dX = (torch.empty(T, inp, dtype=BF16, device="cuda").normal_(generator=g) for _ in range(3))
    A = torch.randn(2, rank, inp, generator=g, device="cuda").mul_(inp ** -0.5).to(BF16)
    B = torch.randn(2, inp, rank, generator=g, device="cuda").to(BF16)
    last = slice(T - 40, T)
    off = torch.tensor([0, T - 20, T], dtype=torch.int32, device="cuda")
    which = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    tail = torch.tensor([0, 20, 40], dtype=torch.int32)
    dY = Y.clone()
    want = dense_ref.adapter(X[last], Y[last], A, B, tail, which, 0.5, dY=dY[last], dX=dX[last])
    Y, H = sn.snack_adapter_forward(X, A, B, off, which, 0.5, Y)
    dX, dA, dB = sn.snack_adapter_backward(X, dY, A, B, off, which, 0.5, H, dX=dX)
    for k, v in (("Y", Y), ("H", H), ("dX", dX)):
        assert_within(k, v[last], *want[k])
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all()
    alone = dense_ref.adapter(X[-20:], Y[-20:], A, B, tail[:2], which[1:], 0.5, dY=dY[-20:])
    assert_within("dA", dA[0], alone["dA"][0][0], alone["dA"][1][0])
    assert_within("dB", dB[0], alone["dB"][0][0], alone["dB"][1][0])
