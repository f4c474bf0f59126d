"""Dropout against its definition: M exact, one rounding of residual + M * x."""

import pytest
import torch

import attention_ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def want(x, p, seed, residual, dtype):
    n = x.numel()
    M = attention_ref.mask_of(seed, torch.zeros(1, dtype=torch.long, device=x.device), n, p).view(x.shape)
    y = torch.where(M == 0, torch.zeros_like(M), x.double() * M)
    return M, y if residual is None else residual.double() + y


def close(got, ref, terms, dtype):
    """Two 32-bit roundings of the terms (2^-24 each, of M and of the product or sum), one of the
    type (float16: magnitudes from 65520 on round to infinity)."""
    u = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
    tiny = 2.0 ** -25 if dtype == F16 else 1e-38
    assert got.dtype == dtype
    err = (got.double() - ref).abs()
    within = (err <= 3 * 2.0 ** -24 * terms + 1.01 * u * ref.abs() + tiny) | (got == ref.to(dtype))
    assert within.all(), float(err.max())


@pytest.mark.parametrize("x_type,y_type", [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (BF16, F32),
                                           (F16, F32), (F32, F16), (BF16, F16), (F16, BF16)])
@pytest.mark.parametrize("shape", [(1,), (3,), (4,), (8,), (9,), (3, 7), (2, 1001), (64, 768), (5, 4099), (300, 4096)])
def test_every_form(x_type, y_type, shape):
    import coo_spmm_sparse_gb300 as sn
    g = torch.Generator(device="cuda").manual_seed(len(shape) + shape[-1])
    x = torch.randn(shape, generator=g, device="cuda").to(x_type)
    r = torch.randn(shape, generator=g, device="cuda").to(y_type)
    for p, seed in ((0.1, 0), (0.5, 2 ** 64 - 1), (0.0, 3), (1e-5, 9), (65535 / 65536, -7)):
        M, y = want(x, p, seed, r, y_type)
        close(sn.snack_dropout_forward(x, p, seed, residual=r), y, r.double().abs() + (x.double() * M).abs(), y_type)
        M, y = want(x, p, seed, None, x_type)
        close(sn.snack_dropout_forward(x, p, seed), y, y.abs(), x_type)
        M, y = want(r, p, seed, None, x_type)
        close(sn.snack_dropout_backward(r, p, seed, dtype=x_type), y, y.abs(), x_type)


def test_mask_is_the_generators():
    import coo_spmm_sparse_gb300 as sn
    y = sn.snack_dropout_forward(torch.ones(1003, device="cuda"), 0.3, 12345)
    T = round(0.3 * 65536)
    for e in (0, 1, 2, 3, 4, 7, 500, 1001, 1002):
        bits = attention_ref.draw(12345, e // 4) >> (16 * (e % 4)) & 0xFFFF
        assert float(y[e]) == (65536 / (65536 - T) if bits >= T else 0.0) or abs(float(y[e]) - 65536 / (65536 - T)) < 1e-6
        assert bool(y[e]) == (bits >= T)


def test_share_and_independence():
    """Means of 2^22 places: within five deviations of p, and of p^2 for two neighbours, rows or seeds."""
    import coo_spmm_sparse_gb300 as sn
    n, p = 1 << 22, 0.1
    x = torch.ones(n, device="cuda")
    drop = [(sn.snack_dropout_forward(x, p, s) == 0).double() for s in (1, 2)]
    q = round(p * 65536) / 65536
    for a, share in ((drop[0], q), (drop[0][1:] * drop[0][:-1], q * q), (drop[0][4:] * drop[0][:-4], q * q),
                     (drop[0] * drop[1], q * q)):
        assert abs(float(a.mean()) - share) <= 5 * (2 * share / n) ** 0.5


def test_dropped_elements_add_nothing():
    import coo_spmm_sparse_gb300 as sn
    x = torch.full((4096,), float("nan"), device="cuda")
    r = torch.arange(4096.0, device="cuda")
    M, _ = want(x, 0.5, 8, None, F32)
    y = sn.snack_dropout_forward(x, 0.5, 8, residual=r)
    assert torch.equal(y[M == 0], r[M == 0]) and y[M != 0].isnan().all()


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_addresses_off_a_vector(shift):
    import coo_spmm_sparse_gb300 as sn
    for dt in (F32, BF16):
        x = torch.randn(5000, device="cuda").to(dt)[shift:]
        r = torch.randn(5000, device="cuda").to(dt)[shift:]
        assert torch.equal(sn.snack_dropout_forward(x, 0.2, 4, residual=r),
                           sn.snack_dropout_forward(x.clone(), 0.2, 4, residual=r.clone()))


def test_autograd_and_differences():
    import coo_spmm_sparse_gb300 as sn
    x = torch.randn(33, 70, device="cuda", requires_grad=True)
    r = torch.randn(33, 70, device="cuda", requires_grad=True)
    dy = torch.randn(33, 70, device="cuda")
    y = sn.snack_dropout(x, 0.25, 6, residual=r)
    y.backward(dy)
    M, ref = want(x.detach(), 0.25, 6, r.detach(), F32)
    assert torch.allclose(x.grad.double(), dy.double() * M, rtol=1e-6)
    assert torch.equal(r.grad, dy)
    # y is linear in x: a difference of any size is its gradient
    u = torch.randn_like(x)
    diff = (sn.snack_dropout_forward(x.detach() + u, 0.25, 6).double() -
            sn.snack_dropout_forward(x.detach(), 0.25, 6).double())
    assert torch.allclose(diff, u.double() * M, atol=1e-5)
    half = torch.randn(4, 8, device="cuda", dtype=BF16, requires_grad=True)
    sn.snack_dropout(half, 0.25, 6, residual=torch.zeros(4, 8, device="cuda")).sum().backward()
    assert half.grad.dtype == BF16
    (g,) = torch.autograd.grad(sn.snack_dropout(x, 0.25, 6).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.sum().backward()


def test_captured_with_a_seed_on_the_device():
    import coo_spmm_sparse_gb300 as sn
    x = torch.randn(1000, device="cuda")
    seed = torch.tensor([5], device="cuda")
    sn.snack_dropout_forward(x, 0.5, seed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sn.snack_dropout_forward(x, 0.5, seed)
        seed.add_(3)
    for step in range(3):
        graph.replay()
        assert torch.equal(y, sn.snack_dropout_forward(x, 0.5, 5 + 3 * step))
    # a seed that changed between forward and backward is noticed
    z = torch.ones(8, device="cuda", requires_grad=True)
    out = sn.snack_dropout(z, 0.5, seed)
    seed.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_refusals():
    import coo_spmm_sparse_gb300 as sn
    x = torch.ones(4, 6, device="cuda")
    f = sn.snack_dropout_forward
    for err, args, opts in [
        (TypeError, (x.cpu(), 0.1, 0), {}), (TypeError, (x.double(), 0.1, 0), {}), (ValueError, (x.t(), 0.1, 0), {}),
        (ValueError, (x, 1.0, 0), {}), (ValueError, (x, -0.1, 0), {}), (ValueError, (x, float("nan"), 0), {}),
        (sn.SnackError, (x, 1 - 2.0 ** -18, 0), {}), (ValueError, (x, 0.1, 0), dict(residual=x[:2])),
        (ValueError, (x, 0.1, 0), dict(residual=x.t().contiguous().t())), (TypeError, (x, 0.1, 0.5), {}),
        (TypeError, (x, 0.1, torch.tensor(1)), {}), (TypeError, (x, 0.1, torch.ones(1, device="cuda")), {}),
    ]:
        with pytest.raises(err):
            f(*args, **opts)
    with pytest.raises(TypeError):
        sn.snack_dropout_backward(x, 0.1, 0, dtype=torch.float64)
    assert f(x[:0], 0.5, 1).shape == (0, 6)
