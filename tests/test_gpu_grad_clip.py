"""The gradient norm over many tensors and clipping, against 64-bit sums.

The norm of n squares is a tree of 32-bit sums of positive terms: held to
1e-5 of its value, and so is the factor; results carry one rounding more."""

import math

import pytest
import torch

from dense_ref import assert_within

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def tensors(sizes, types, seed=0, std=0.1, offset=0):
    """One tensor per size; offset: elements by which each starts off a 16-byte boundary."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        k = offset * (i % 5)
        t = (torch.randn(n + k, generator=g, device="cuda") * std).to(types[i % len(types)])
        out.append(t[k:])
    return out


def norm64(ts, kind):
    v = [t.double() for t in ts if t.numel()]
    if not v:
        return 0.0
    if kind == math.inf:
        return float(torch.stack([t.abs().max() for t in v]).max())
    return float(torch.stack([t.square().sum() for t in v]).sum().sqrt())


LISTS = [
    ([1], [F32], 0),
    ([5, 1, 0, 33, 4096, 70001], [F32], 0),
    ([5, 1, 0, 33, 4096, 70001], [F32, BF16, F16], 1),
    ([1000] * 148 + [3_000_001], [F32], 0),
    ([777] * 300, [BF16, F32], 3),
    ([17 + (i * 37) % 900 for i in range(2500)], [F32, F16], 1),
    ([5_000_003, 9_000_000], [BF16], 1),
]


@pytest.mark.parametrize("sizes,types,offset", LISTS)
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_norm(sizes, types, offset, kind):
    import coo_spmm_sparse_gb300 as sn
    ts = tensors(sizes, types, 1, offset=offset)
    want = norm64(ts, kind)
    for g in (ts, sn.snack_tensor_list(ts)):
        got = float(sn.snack_grad_norm(g, kind))
        assert abs(got - want) <= 1e-5 * want


@pytest.mark.parametrize("sizes,types,offset", LISTS)
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("share", [0.3, 1.7])
def test_clip_in_place(sizes, types, offset, kind, share):
    import coo_spmm_sparse_gb300 as sn
    ts = tensors(sizes, types, 2, offset=offset)
    before = [t.clone() for t in ts]
    want = norm64(ts, kind)
    got = float(sn.snack_clip_grad_norm(ts, share * want, kind))
    assert abs(got - want) <= 1e-5 * want
    coef = min(1.0, share * want / (want + 1e-6))
    for t, b in zip(ts, before):
        if coef == 1.0:
            assert torch.equal(t, b)
        else:
            v = b.double() * coef
            assert_within("clipped", t, v, 2 * v.abs())


@pytest.mark.parametrize("sizes,types,offset", LISTS)
@pytest.mark.parametrize("dst,shift", [(F32, 0), (F32, 1), (BF16, 0), (BF16, 3), (F16, 1)])
@pytest.mark.parametrize("share", [0.3, 1.7])
def test_clip_into_other_tensors(sizes, types, offset, dst, shift, share):
    import coo_spmm_sparse_gb300 as sn
    ts = tensors(sizes, types, 3, offset=offset)
    # packed end to end, `shift` elements off a 16-byte boundary, between guards
    flat = torch.full((sum(sizes) + 64 + shift,), 7.0, dtype=dst, device="cuda")
    out, at = [], 32 + shift
    for n in sizes:
        out.append(flat[at: at + n])
        at += n
    want = norm64(ts, 2.0)
    before = [t.clone() for t in ts]
    got = float(sn.snack_clip_grad_norm(ts, share * want, out=out))
    assert abs(got - want) <= 1e-5 * want
    coef = min(1.0, share * want / (want + 1e-6))
    for t, b, o in zip(ts, before, out):
        assert torch.equal(t, b)
        v = b.double() * coef
        assert_within("clipped", o, v, 2 * v.abs())
    assert (flat[: 32 + shift] == 7).all() and (flat[at:] == 7).all()


def test_nothing_and_zeros():
    import coo_spmm_sparse_gb300 as sn
    assert float(sn.snack_grad_norm([])) == 0.0
    assert float(sn.snack_clip_grad_norm([], 1.0)) == 0.0
    z = [torch.zeros(10, device="cuda"), torch.zeros(0, device="cuda")]
    for kind in (2.0, math.inf):
        assert float(sn.snack_grad_norm(z, kind)) == 0.0
    assert float(sn.snack_clip_grad_norm(z, 0.0)) == 0.0
    assert torch.equal(z[0], torch.zeros(10, device="cuda"))
    e = [torch.zeros(0, device="cuda")]
    assert float(sn.snack_clip_grad_norm(e, 1.0)) == 0.0


@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("where", [0, 100_002])
def test_nan_and_infinity(kind, where):
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([100_003, 50], [F32, BF16], 4)
    ts[0][where] = float("inf")
    assert float(sn.snack_grad_norm(ts, kind)) == math.inf
    sn.snack_clip_grad_norm(ts, 1.0, kind)  # inf * 0 is NaN, what is finite becomes 0
    assert torch.isnan(ts[0][where]) and float(ts[0].nan_to_num(0.0).abs().sum()) == 0.0
    ts = tensors([100_003, 50], [F32, BF16], 4)
    ts[0][where] = float("nan")
    assert math.isnan(float(sn.snack_grad_norm(ts, kind)))
    sn.snack_clip_grad_norm(ts, 1.0, kind)
    assert torch.isnan(ts[0]).all() and torch.isnan(ts[1]).all()


def test_matches_torch_on_a_model_and_keeps_bits():
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([768 * 50, 768, 3, 100_001] * 9, [F32], 5)
    ps = [torch.nn.Parameter(torch.zeros_like(t)) for t in ts]
    for p, t in zip(ps, ts):
        p.grad = t.clone()
    want = torch.nn.utils.clip_grad_norm_(ps, 1.0)
    runs = []
    for _ in range(3):
        mine = [t.clone() for t in ts]
        runs.append((float(sn.snack_clip_grad_norm(mine, 1.0)), mine))
    assert abs(runs[0][0] - float(want)) <= 1e-5 * float(want)
    for p, m in zip(ps, runs[0][1]):
        assert torch.allclose(p.grad, m, rtol=2e-5, atol=0)
    for n, m in runs[1:]:
        assert n == runs[0][0] and all(torch.equal(a, b) for a, b in zip(m, runs[0][1]))


def test_other_stream_and_graph():
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([100_000, 7, 4096], [F32], 6)
    want = norm64(ts, 2.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n1 = sn.snack_grad_norm(ts, stream=s)
    s.synchronize()
    assert abs(float(n1) - want) <= 1e-5 * want
    lst, out = sn.snack_tensor_list(ts), [torch.empty_like(t) for t in ts]
    norm = torch.zeros((), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sn.snack_clip_grad_norm(lst, 1.0, out=out, norm=norm)
    for t in ts:
        t.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - 2 * want) <= 2e-5 * want
    for t, o in zip(ts, out):
        v = t.double() / (2 * want + 1e-6)
        assert_within("clipped", o, v, 2 * v.abs())


def test_refusals():
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([10, 20], [F32])
    with pytest.raises(TypeError):
        sn.snack_grad_norm([ts[0].cpu()])
    with pytest.raises(TypeError):
        sn.snack_grad_norm([ts[0].double()])
    with pytest.raises(ValueError):
        sn.snack_grad_norm([torch.zeros(4, 6, device="cuda").t()])
    with pytest.raises(ValueError):
        sn.snack_grad_norm(ts, 1.0)
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError):
            sn.snack_clip_grad_norm(ts, bad)
    with pytest.raises(ValueError):
        sn.snack_clip_grad_norm(ts, 1.0, out=[ts[0]])
    with pytest.raises(ValueError):
        sn.snack_clip_grad_norm(ts, 1.0, out=[ts[1], ts[0]])
    with pytest.raises(ValueError):
        sn.snack_grad_norm(ts, norm=torch.zeros(2, device="cuda"))
    with pytest.raises(sn.SnackError) as e:
        sn.snack_clip_grad_norm(ts, 1.0, eps=-1.0)
    assert e.value.status == 1


def test_tensors_that_only_the_call_holds():
    """A generator's tensors live until the call has launched its work: their
    memory is not handed out for the call's own scratch or result."""
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([1000 + 64 * i for i in range(40)], [F32], 8)
    want = norm64([t * 3 for t in ts], 2.0)
    for _ in range(3):
        got = float(sn.snack_grad_norm(t * 3 for t in ts))
        assert abs(got - want) <= 1e-5 * want
        out = [torch.empty_like(t) for t in ts]
        got = float(sn.snack_clip_grad_norm((t * 3 for t in ts), 0.5 * want, out=iter(out)))
        assert abs(got - want) <= 1e-5 * want
        for t, o in zip(ts, out):
            v = t.double() * 3 * 0.5 * want / (want + 1e-6)
            assert_within("clipped", o, v, 2 * v.abs())


def test_kept_list_follows_its_tensors():
    """A kept list means its tensors, not the memory that they had when it
    was made: new storage, type or size is seen by the next call."""
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([4096, 70_001, 5], [F32], 9)
    kept = sn.snack_tensor_list(ts)
    old = [t.clone() for t in ts]
    held = ts[1].data  # the memory of before stays somebody else's
    ts[0].data = torch.full((4096,), 2.0, device="cuda")        # other memory
    ts[1].data = (ts[1].data * 0.5).bfloat16()                  # another type
    with torch.no_grad():
        ts[2].set_(torch.full((9,), 3.0, device="cuda"))        # another size
    want = norm64(ts, 2.0)
    assert abs(float(sn.snack_grad_norm(kept)) - want) <= 1e-5 * want
    before = [t.clone() for t in ts]
    sn.snack_clip_grad_norm(kept, 0.25 * want)
    for t, b in zip(ts, before):
        v = b.double() * 0.25 * want / (want + 1e-6)
        assert_within("clipped", t, v, 2 * v.abs())
    assert torch.equal(held, old[1])
    out = sn.snack_tensor_list([torch.empty_like(t) for t in ts])
    sn.snack_clip_grad_norm(kept, 1.0, out=out)
    ts[0].data = torch.ones(7, device="cuda")
    with pytest.raises(ValueError, match="as many elements"):
        sn.snack_clip_grad_norm(kept, 1.0, out=out)
    ts[0].data = torch.ones(4, 6, device="cuda").t()
    with pytest.raises(ValueError, match="contiguous"):
        sn.snack_grad_norm(kept)
    ts[0].data = torch.ones(6, device="cuda", dtype=torch.float64)
    with pytest.raises(TypeError):
        sn.snack_grad_norm(kept)


def test_empty_tensors_after_a_full_table():
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([40] * 1024 + [0] * 1030 + [3], [F32], 12)
    for gs in (ts, ts[:-1]):
        want = norm64(gs, 2.0)
        before = [t.clone() for t in gs]
        assert abs(float(sn.snack_clip_grad_norm(gs, 0.5 * want)) - want) <= 1e-5 * want
        for t, b in zip(gs, before):
            v = b.double() * 0.5 * want / (want + 1e-6)
            assert_within("clipped", t, v, 2 * v.abs())


def test_writes_in_place_are_seen_by_autograd():
    """A tensor that autograd keeps for a backward pass and a call then
    changes: the backward pass raises, it does not use the changed values."""
    import coo_spmm_sparse_gb300 as sn
    g, o = torch.randn(64, device="cuda"), torch.randn(64, device="cuda")
    norm = torch.ones((), device="cuda")
    kept = sn.snack_tensor_list([g])
    for changed, call in ((g, lambda: sn.snack_clip_grad_norm([g], 1e-3)),
                          (o, lambda: sn.snack_clip_grad_norm(kept, 1.0, out=[o])),
                          (norm, lambda: sn.snack_grad_norm(kept, norm=norm))):
        w = torch.ones(changed.shape, device="cuda", requires_grad=True)
        z = (changed * w).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.backward()
    with torch.inference_mode():  # tensors without a version
        g = torch.ones(64, device="cuda")
        sn.snack_clip_grad_norm([g], 1.0)
        assert abs(float(g[0]) - 1 / 8) <= 1e-5


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-25, 1e-18, 1e-15, 1e18, 1e25, 1e35])
def test_magnitudes_whose_squares_leave_the_range(dt, size):
    """The norm of finite gradients is theirs wherever it is a float32
    itself, and clipping scales them by it."""
    import coo_spmm_sparse_gb300 as sn
    ts = tensors([5, 4096, 70_001], [dt], 11, std=1.0, offset=1)
    for mixed in (False, True):
        gs = [(t.double() * size).to(dt) for t in ts]
        if mixed:  # among gradients of ordinary size
            gs[1] = ts[1] * 1e-3
        want = norm64(gs, 2.0)
        got = float(sn.snack_grad_norm(gs))
        assert abs(got - want) <= 1e-5 * want
        before = [t.clone() for t in gs]
        sn.snack_clip_grad_norm(gs, 0.5 * want, eps=0.0)
        for t, b in zip(gs, before):
            v = b.double() * 0.5
            # float32 and bfloat16 below 2^-126 keep no more than half their last bit
            tiny = 2.0 ** -149 if dt == F32 else 2.0 ** -134
            err = (t.double() - v).abs()
            assert bool((err <= (1e-5 + (2.0 ** -8 if dt == BF16 else 0)) * v.abs() + tiny).all())


def test_a_norm_beyond_float32():
    """Finite gradients whose norm no float32 holds: the norm is infinite,
    the factor is not lost."""
    import coo_spmm_sparse_gb300 as sn
    g = torch.full((4096,), 3e38, device="cuda")
    assert float(sn.snack_grad_norm([g])) == math.inf
    sn.snack_clip_grad_norm([g], 1e30)
    want = 1e30 / 64
    assert bool(((g.double() - want).abs() <= 1e-5 * want).all())


def test_what_runs_next_keeps_its_cache():
    """A kernel that reads 96 MB from the L2 again and again is no slower after
    a norm than after any other read of the gradients (evicted last, 64 MB of
    them made it a third slower, and stayed).  Medians of 20, the best of five."""
    import coo_spmm_sparse_gb300 as sn
    ts = [t for t in torch.randn(40_000_000, device="cuda").bfloat16().split(400_000)]
    kept, w = sn.snack_tensor_list(ts), torch.randn(24_000_000, device="cuda")

    def after(call):
        times = []
        for _ in range(20):
            call()
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            for _ in range(4):
                torch.sum(w)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[10]

    flat = ts[0].as_strided((40_000_000,), (1,))
    plain = min(after(lambda: torch.sum(flat)) for _ in range(3))
    ratios = []
    for call in (lambda: sn.snack_grad_norm(kept), lambda: sn.snack_clip_grad_norm(kept, 1e9)):
        ratios.append(min(after(call) for _ in range(5)) / plain)
    assert max(ratios) <= 1.15, ratios


def test_offsets_beyond_32_bits():
    import coo_spmm_sparse_gb300 as sn
    n = 2 ** 31 + 70_001
    t = torch.full((n,), 0.5, dtype=BF16, device="cuda")
    t[-1] = 256.0
    want = math.sqrt((n - 1) * 0.25 + 65536.0)
    got = float(sn.snack_clip_grad_norm([t], 0.5 * want))
    assert abs(got - want) <= 1e-5 * want
    assert float(t[-1]) == 128.0 and float(t[0]) == float(t[-2]) == 0.25
    assert float(t[2 ** 31 - 5: 2 ** 31 + 5].float().sum()) == 2.5
