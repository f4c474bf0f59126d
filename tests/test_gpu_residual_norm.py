"""The block norms with gate and residual scales against a 64-bit evaluation
of their definition (bounds in dense_ref.py), their gradients also against
differences, and what the calls refuse."""

import pytest
import torch

import dense_ref
from dense_ref import assert_within

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (F32, F16)]


def make(shape, kind, post, gate, stream, branch, param=F32, seed=0, offset=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = shape[-1]

    def rnd(s, std=1.0, mean=0.0, dt=F32):
        return (torch.randn(s, generator=g, device="cuda") * std + mean).to(dt)

    x, y = rnd(shape, 2.0, offset, stream), rnd(shape, 0.7, offset, branch)
    gshape = {None: None, "channel": (d,), "token": (*shape[:-1], 1),
              "sequence": (*shape[:-2], 1, d), "full": shape}[gate]
    o = dict(kind=kind, post_norm=post, residual_scale=0.9, branch_scale=0.7, eps=1e-5,
             gate=None if gshape is None else rnd(gshape, 0.5, 0.6, branch),
             next_weight=rnd((d,), 0.2, 1.0, param))
    if kind == "layer":
        o["next_bias"] = rnd((d,), 0.2, 0.0, param)
    if post:
        o["post_weight"] = rnd((d,), 0.2, 1.0, param)
        if kind == "layer":
            o["post_bias"] = rnd((d,), 0.2, 0.0, param)
    return x, y, o, rnd(shape, 1.0, 0.0, stream), rnd(shape, 1.0, 0.0, branch)


def check(x, y, o, dr, dh):
    import coo_spmm_sparse_gb300 as sn
    r, h, stats = sn.snack_residual_norm_forward(x, y, **o)
    got = {"r": r, "h": h}
    got.update(sn.snack_residual_norm_backward(dr, dh, x, y, stats, **o))
    torch.cuda.synchronize()
    want = dense_ref.residual_norm(x, y, dr=dr, dh=dh, **o)
    for k, (v, S) in want.items():
        if got[k] is not None:
            assert_within(k, got[k], v, S)
    return got


@pytest.mark.parametrize("stream,branch", TYPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token", "sequence", "full"])
def test_every_form(stream, branch, kind, post, gate):
    check(*make((3, 37, 256), kind, post, gate, stream, branch, seed=1))


@pytest.mark.parametrize("d", [1, 2, 7, 33, 64, 100, 255, 768, 1000, 1001, 1024, 2304, 4096, 4100,
                               5003, 8192, 8200, 12288, 16384, 20001,
                               32768, 33000, 40001])
@pytest.mark.parametrize("stream,branch", [(F32, F32), (BF16, BF16), (F32, BF16)])
def test_every_width(d, stream, branch):
    kind = "layer" if d > 1 else "rms"  # a layer norm of one element is its bias
    check(*make((1, 5, d), kind, True, "channel", stream, branch, seed=d))
    check(*make((2, 3, d), "rms", False, "sequence", stream, branch, seed=d + 1))


@pytest.mark.parametrize("rows", [1, 2, 31, 255, 1024, 4099])
@pytest.mark.parametrize("gate", [None, "channel", "sequence"])
def test_every_length(rows, gate):
    check(*make((1, rows, 768), "layer", False, gate, F32, F32, seed=rows))
    check(*make((rows, 1, 512), "rms", True, gate, BF16, BF16, seed=rows))


@pytest.mark.parametrize("param", [F32, BF16])
def test_parameters_in_sixteen_bits(param):
    check(*make((2, 65, 640), "layer", True, "channel", F32, BF16, param=param, seed=4))


def test_biases_of_an_rms_norm():
    for stream, branch in ((F32, F32), (BF16, BF16)):
        for gate in (None, "channel", "sequence", "token", "full"):
            x, y, o, dr, dh = make((2, 33, 264), "layer", True, gate, stream, branch, seed=21)
            check(x, y, dict(o, kind="rms"), dr, dh)


def test_strided_rows_and_misaligned_starts():
    for d, off in ((256, 0), (256, 3), (768, 8), (100, 1)):
        x, y, o, dr, dh = make((2, 9, d), "layer", True, "full", BF16, BF16, seed=9)
        big = torch.zeros(2, 9, d + 24, dtype=BF16, device="cuda")

        def wide(t, at):
            v = torch.zeros_like(big)[..., at: at + d]
            v.copy_(t)
            return v

        got = check(wide(x, off), wide(y, off), dict(o, gate=wide(o["gate"], off)), wide(dr, off),
                    wide(dh, 0))
        ref = check(x, y, o, dr, dh)
        assert got["r"].shape == ref["r"].shape


def test_plain_norm_without_a_branch():
    import coo_spmm_sparse_gb300 as sn
    for stream, branch in TYPES:
        x, _, o, dr, dh = make((3, 11, 320), "layer", False, None, stream, branch, seed=5)
        o.update(residual_scale=1.0, branch_scale=1.0)
        r, h, stats = sn.snack_residual_norm_forward(x, None, branch_dtype=branch, **o)
        assert r is x and h.dtype == branch
        g = sn.snack_residual_norm_backward(dr, dh, x, None, stats, branch_dtype=branch, **o)
        assert "dy" not in g
        want = dense_ref.residual_norm(x, None, dr=dr, dh=dh, **o)
        for k, v in dict(g, h=h).items():
            assert_within(k, v, *want[k])


def test_missing_gradients_and_no_next_norm():
    import coo_spmm_sparse_gb300 as sn
    x, y, o, dr, dh = make((2, 9, 256), "rms", True, "channel", F32, F32, seed=6)
    _, _, stats = sn.snack_residual_norm_forward(x, y, **o)
    for a, b in ((dr, None), (None, dh)):
        g = sn.snack_residual_norm_backward(a, b, x, y, stats, **o)
        want = dense_ref.residual_norm(x, y, dr=a, dh=b, **o)
        for k, v in g.items():
            assert_within(k, v, *want[k])
    o = dict(o, next_norm=False, next_weight=None)
    r, h, stats = sn.snack_residual_norm_forward(x, y, **o)
    assert h is None
    g = sn.snack_residual_norm_backward(dr, None, x, y, stats, **o)
    want = dense_ref.residual_norm(x, y, dr=dr, **o)
    for k, v in dict(g, r=r).items():
        assert_within(k, v, *want[k])


def test_rows_of_equal_elements_and_zero_rows():
    # variance 0: 1 / sqrt(eps) multiplies exact zeros
    import coo_spmm_sparse_gb300 as sn
    x = torch.zeros(3, 128, device="cuda")
    x[1] = 2.0
    r, h, _ = sn.snack_residual_norm_forward(x, torch.zeros_like(x))
    assert torch.equal(r, x) and torch.equal(h, torch.zeros_like(x))
    _, h, _ = sn.snack_residual_norm_forward(x, torch.zeros_like(x), kind="rms")
    assert torch.equal(h[0], torch.zeros(128, device="cuda"))
    assert_within("h", h[1], torch.full((128,), 2.0 / (4.0 + 1e-5) ** 0.5, dtype=torch.float64),
                  torch.ones(128))


def test_nan_and_infinity_stay_in_their_row():
    import coo_spmm_sparse_gb300 as sn
    x, y, o, _, _ = make((1, 6, 300), "layer", True, "channel", F32, F32, seed=7)
    ref = sn.snack_residual_norm_forward(x, y, **o)[1].clone()
    x[0, 2, 17], x[0, 4, 5] = float("nan"), float("inf")
    r, h, _ = sn.snack_residual_norm_forward(x, y, **o)
    assert torch.isnan(h[0, 2]).all() and torch.isnan(h[0, 4]).any()
    for i in (0, 1, 3, 5):
        assert torch.equal(h[0, i], ref[0, i])


def test_no_rows():
    import coo_spmm_sparse_gb300 as sn
    x, y, o, dr, dh = make((1, 4, 64), "layer", True, "channel", F32, F32, seed=8)
    x, y, dr, dh = (t[:, :0] for t in (x, y, dr, dh))
    r, h, stats = sn.snack_residual_norm_forward(x, y, **o)
    assert r.shape == h.shape == (1, 0, 64)
    g = sn.snack_residual_norm_backward(dr, dh, x, y, stats, **o)
    for k in ("dgate", "dpost_weight", "dpost_bias", "dnext_weight", "dnext_bias"):
        assert torch.equal(g[k], torch.zeros(64, device="cuda")), k


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("gate", ["channel", "token", "sequence", "full"])
def test_gradients_against_differences(kind, gate):
    """d/de of sum(r cr + h ch) along a random direction.  Step 1e-2: the
    central difference is off by O(1e-4) of third derivatives and by the
    rounding of the sums (2^-24 * ~800 terms / 2e-2 = 2e-3); the derivative
    is a sum of ~400 terms of order 1, held to 1 % of their 2-norm."""
    import coo_spmm_sparse_gb300 as sn
    x, y, o, cr, ch = make((2, 4, 48), kind, True, gate, F32, F32, seed=11)
    _, _, stats = sn.snack_residual_norm_forward(x, y, **o)
    g = sn.snack_residual_norm_backward(cr, ch, x, y, stats, **o)
    gen = torch.Generator(device="cuda").manual_seed(3)
    names = {"dx": None, "dy": None, "dgate": "gate", "dpost_weight": "post_weight",
             "dnext_weight": "next_weight"}
    for k, opt in names.items():
        base = {"dx": x, "dy": y}.get(k, o.get(opt))
        e = torch.randn(base.shape, generator=gen, device="cuda")
        loss = []
        for step in (1e-2, -1e-2):
            v = base + step * e
            xx, yy, oo = (v if k == "dx" else x), (v if k == "dy" else y), dict(o)
            if opt:
                oo[opt] = v
            r, h, _ = sn.snack_residual_norm_forward(xx, yy, **oo)
            loss.append((r.double() * cr.double() + h.double() * ch.double()).sum())
        got = float((g[k].double() * e.double()).sum())
        want = float(loss[0] - loss[1]) / 2e-2
        scale = float((g[k].double() * e.double()).norm())
        assert abs(got - want) <= 1e-2 * (scale + 1.0), (k, got, want, scale)


def test_module_matches_autograd_of_the_definition():
    import coo_spmm_sparse_gb300 as sn
    torch.manual_seed(0)
    m = sn.SnackResidualNorm(192, kind="layer", post=True, gate="channel", gate_init=0.5,
                             branch_scale=0.8)
    x = torch.randn(2, 7, 192, device="cuda", requires_grad=True)
    y = torch.randn(2, 7, 192, device="cuda", requires_grad=True)
    c = torch.randn(192, device="cuda")
    r, h = m(x, y)
    (r.square().sum() + (h * c).sum(-1).square().sum()).backward()
    got = {"x": x.grad, "y": y.grad, **{k: p.grad for k, p in m.named_parameters()}}
    x64, y64 = (t.detach().double().requires_grad_() for t in (x, y))
    p = {k: v.detach().double().requires_grad_() for k, v in m.named_parameters()}
    ln = torch.nn.functional.layer_norm
    rr = x64 + 0.8 * p["gate"] * ln(y64, (192,), p["post_weight"], p["post_bias"], 1e-5)
    hh = ln(rr, (192,), p["next_weight"], p["next_bias"], 1e-5)
    (rr.square().sum() + (hh * c.double()).sum(-1).square().sum()).backward()
    for k, v in {"x": x64, "y": y64, **p}.items():
        scale = v.grad.abs().max()
        assert torch.allclose(got[k].double(), v.grad, rtol=1e-4, atol=1e-5 * float(scale)), k


def test_plain_norm_carries_both_gradients():
    import coo_spmm_sparse_gb300 as sn
    torch.manual_seed(1)
    x = torch.randn(3, 5, 160, device="cuda", requires_grad=True)
    w = torch.randn(160, device="cuda", requires_grad=True)
    c1, c2 = torch.randn(2, 3, 5, 160, device="cuda")
    r, h = sn.snack_residual_norm(x, next_weight=w, kind="layer")
    ((r * c1).sum() + (h * c2).sum()).backward()
    x64, w64 = (t.detach().double().requires_grad_() for t in (x, w))
    hh = torch.nn.functional.layer_norm(x64, (160,), w64, None, 1e-5)
    ((x64 * c1.double()).sum() + (hh * c2.double()).sum()).backward()
    assert torch.equal(r, x)
    for got, want in ((x.grad, x64.grad), (w.grad, w64.grad)):
        assert torch.allclose(got.double(), want, rtol=1e-4, atol=1e-5 * float(want.abs().max()))
    # only one of the two is used
    x.grad = None
    sn.snack_residual_norm(x, next_weight=w)[1].square().sum().backward()
    assert x.grad is not None


def test_mixed_types_through_the_module():
    import coo_spmm_sparse_gb300 as sn
    torch.manual_seed(2)
    m = sn.SnackResidualNorm(256, kind="rms", post=True, gate="channel", gate_init=0.25)
    x = torch.randn(2, 6, 256, device="cuda", requires_grad=True)
    y = torch.randn(2, 6, 256, device="cuda").bfloat16().requires_grad_()
    r, h = m(x, y)
    assert r.dtype == F32 and h.dtype == BF16
    (r.sum() + h.float().square().sum()).backward()
    assert x.grad.dtype == F32 and y.grad.dtype == BF16 and m.gate.grad.dtype == F32
    want = dense_ref.residual_norm(x, y, kind="rms", post_norm=True, post_weight=m.post_weight,
                                   gate=m.gate.detach().bfloat16(), next_weight=m.next_weight,
                                   dr=torch.ones_like(x), dh=(2 * h.detach().float()).bfloat16())
    for got, k in ((x.grad, "dx"), (y.grad, "dy"), (m.next_weight.grad, "dnext_weight")):
        assert_within(k, got, *want[k])


def test_same_bits_every_time_and_on_another_stream():
    import coo_spmm_sparse_gb300 as sn
    x, y, o, dr, dh = make((4, 513, 768), "rms", True, "sequence", BF16, BF16, seed=12)
    r, h, stats = sn.snack_residual_norm_forward(x, y, **o)
    first = sn.snack_residual_norm_backward(dr, dh, x, y, stats, **o)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r2, h2, stats2 = sn.snack_residual_norm_forward(x, y, **o)
        again = sn.snack_residual_norm_backward(dr, dh, x, y, stats2, **o)
    torch.cuda.synchronize()
    assert torch.equal(r, r2) and torch.equal(h, h2)
    for k in first:
        assert torch.equal(first[k], again[k]), k


def test_refusals():
    import coo_spmm_sparse_gb300 as sn
    x, y, o, dr, dh = make((2, 3, 64), "layer", False, None, F32, F32)
    f = sn.snack_residual_norm_forward
    with pytest.raises(TypeError):
        f(x.cpu(), y)
    with pytest.raises(TypeError):
        f(x.double(), y)
    with pytest.raises(TypeError):
        f(x.bfloat16(), y)  # the residual stream in fewer bits than the branch
    with pytest.raises(ValueError):
        f(x, y[..., :32])
    with pytest.raises(ValueError):
        f(x, y, kind="group")
    with pytest.raises(ValueError):
        f(x, None, post_norm=True)
    with pytest.raises(ValueError):
        f(x, y, post_weight=o["next_weight"])
    with pytest.raises(ValueError):
        f(x, y, gate=torch.ones(3, 1, device="cuda"))
    with pytest.raises(ValueError):
        f(x, y, next_weight=o["next_weight"][:5])
    with pytest.raises(ValueError):
        f(x.transpose(1, 2), y.transpose(1, 2))
    with pytest.raises(sn.SnackError) as e:
        f(x, y, eps=-1.0)
    assert e.value.status == 1
    _, _, stats = f(x, y)
    with pytest.raises(ValueError):
        sn.snack_residual_norm_backward(dr, dh[..., :3], x, y, stats)
    with pytest.raises(ValueError):
        sn.snack_residual_norm_backward(dr, dh, x, y, stats[:1])
    with pytest.raises(ValueError):
        sn.snack_residual_norm_backward(dr, dh, x, y, stats, next_norm=False)


@pytest.mark.parametrize("stream,branch", [(F32, F32), (F32, BF16)])
def test_gate_of_sequences_without_rows(stream, branch):
    """Sequences of no rows: their gates have no terms, so their gradient is zero."""
    import coo_spmm_sparse_gb300 as sn
    x, y, o, dr, dh = make((2, 4, 64), "layer", True, "sequence", stream, branch, seed=13)
    x, y, dr, dh = (t[:, :0] for t in (x, y, dr, dh))
    _, _, stats = sn.snack_residual_norm_forward(x, y, **o)
    for n in (64, 128):  # what the allocator hands out next holds no zeros
        junk = [torch.full((n,), float("nan"), device="cuda") for _ in range(16)]
        del junk
    g = sn.snack_residual_norm_backward(dr, dh, x, y, stats, **o)
    assert torch.equal(g["dgate"], torch.zeros(2, 1, 64, dtype=branch, device="cuda"))
    for k in ("dpost_weight", "dpost_bias", "dnext_weight", "dnext_bias"):
        assert torch.equal(g[k], torch.zeros(64, device="cuda")), k


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token", "sequence", "full"])
@pytest.mark.parametrize("d", [256, 250, 33000])
def test_gradients_of_biases_that_are_not_there(kind, post, gate, d):
    """The C call writes every gradient it is asked for: that of a bias left
    out (NULL: zero) is the same sum as that of a bias of zeros."""
    import dense_abi as abi
    x, y, o, dr, dh = make((3, 5, d), kind, post, gate, F32, F32, seed=14)
    zeros = torch.zeros(d, device="cuda")
    o["next_bias"] = zeros
    if post:
        o["post_bias"] = zeros
    want = dense_ref.residual_norm(x, y, dr=dr, dh=dh, **o)
    rows = [t.reshape(15, d) for t in (x, y, dr, dh)]
    stats, r, h = torch.empty(15, 4, device="cuda"), torch.empty_like(rows[0]), torch.empty_like(rows[0])
    opts = {k: v for k, v in o.items() if k not in ("next_bias", "post_bias")}
    a = abi.norm_args(*rows[:2], stats, gate_kind=gate, group_rows=5 if gate == "sequence" else 0,
                      **opts)
    assert abi.norm_forward(a, r, h) == 0
    names = ["dnext_weight", "dnext_bias"] + (["dpost_weight", "dpost_bias"] if post else [])
    got = {k: torch.full((d,), float("nan"), device="cuda") for k in names}
    got.update(dx=torch.empty_like(r), dy=torch.empty_like(r))
    assert abi.norm_backward(a, dr=rows[2], dh=rows[3], **got) == 0
    torch.cuda.synchronize()
    for k, v in got.items():
        assert_within(k, v.reshape(want[k][0].shape), *want[k])


@pytest.mark.parametrize("d", [256, 33000])
def test_what_belongs_to_no_option_is_refused(d):
    """Weights, biases and gradients of a norm, gate or branch that is not
    there: refused by the C calls at every width."""
    import dense_abi as abi
    x, y = torch.randn(2, 3, d, device="cuda")
    w, stats = torch.ones(d, device="cuda"), torch.empty(3, 4, device="cuda")
    r, h, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    for name in ("post_weight", "post_bias"):
        assert abi.norm_forward(abi.norm_args(x, y, stats, **{name: w}), r, h) == abi.INVALID_ARG
        assert name[5:] in abi.lib().snack_last_error(None).decode()
    for name in ("next_weight", "next_bias"):
        a = abi.norm_args(x, y, stats, next_norm=0, **{name: w})
        assert abi.norm_forward(a, r, None) == abi.INVALID_ARG
    a = abi.norm_args(x, y, stats)
    assert abi.norm_forward(a, r, h) == 0
    for name in ("dpost_weight", "dpost_bias", "dgate"):
        assert abi.norm_backward(a, dr=x, dh=y, dx=dx, **{name: w}) == abi.INVALID_ARG
    a.next_norm = 0
    for grads in (dict(dnext_weight=w), dict(dnext_bias=w), dict(dh=y)):
        assert abi.norm_backward(a, dr=x, dx=dx, **grads) == abi.INVALID_ARG
    a = abi.norm_args(x, None, stats)
    assert abi.norm_forward(a, r, h) == 0
    assert abi.norm_backward(a, dr=x, dh=y, dx=dx, dy=r) == abi.INVALID_ARG
    assert abi.norm_backward(a, dr=x, dh=y, dx=dx) == 0


def test_calls_of_two_host_threads():
    """The C calls run from any host thread: two threads at widths whose
    kernels take unlike amounts of shared memory do not disturb each other."""
    import threading
    import dense_abi as abi
    widths, failed = (4096, 2048), []
    start = threading.Barrier(2)

    def work(d):
        s = torch.cuda.Stream()
        x, y, stats = torch.randn(2, d, device="cuda"), torch.randn(2, d, device="cuda"), \
            torch.empty(2, 4, device="cuda")
        r, h = torch.empty_like(x), torch.empty_like(x)
        torch.cuda.synchronize()
        a = abi.norm_args(x, y, stats)
        start.wait()
        for _ in range(20000):
            st = abi.norm_forward(a, r, h, s.cuda_stream)
            if st != 0:
                failed.append((d, st, abi.lib().snack_last_error(None)))
                return
        s.synchronize()

    threads = [threading.Thread(target=work, args=(d,)) for d in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_second_derivatives_raise():
    """The backward's results carry no graph: differentiating them again
    raises, whatever the incoming gradient, where a constant would be wrong."""
    import coo_spmm_sparse_gb300 as sn
    for loss in (lambda r, h: h.sum(), lambda r, h: (r * h).sum()):
        x = torch.randn(3, 64, device="cuda", requires_grad=True)
        y = torch.randn(3, 64, device="cuda", requires_grad=True)
        w = torch.ones(64, device="cuda", requires_grad=True)
        for i, t in enumerate((x, y, w)):
            r, h = sn.snack_residual_norm(x, y, next_weight=w)
            g, = torch.autograd.grad(loss(r, h), t, create_graph=True)
            with pytest.raises(RuntimeError, match="second derivative"):
                (h.sum() + g.square().sum()).backward()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows are as they are alone."""
    import coo_spmm_sparse_gb300 as sn
    rows, d = 66_000, 32_768
    g = torch.Generator(device="cuda").manual_seed(15)
    x, y, dr, dh = (torch.empty(1, rows, d, dtype=BF16, device="cuda").normal_(generator=g)
                    for _ in range(4))
    o = dict(kind="rms", post_norm=True, gate=torch.rand(1, rows, 1, device="cuda").to(BF16),
             next_weight=torch.rand(d, generator=g, device="cuda"))
    r, h, stats = sn.snack_residual_norm_forward(x, y, **o)
    got = dict(sn.snack_residual_norm_backward(dr, dh, x, y, stats, **o), r=r, h=h)
    last = slice(rows - 3, rows)
    tail = [t[:, last].contiguous() for t in (x, y, dr, dh)]
    want = dense_ref.residual_norm(*tail[:2], dr=tail[2], dh=tail[3],
                                   **dict(o, gate=o["gate"][:, last]))
    for k in ("r", "h", "dx", "dy", "dgate"):
        assert_within(k, got[k][:, last], *want[k])
