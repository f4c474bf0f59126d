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
