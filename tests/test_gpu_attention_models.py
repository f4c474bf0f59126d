"""The decoders around the attention and the dropout: sizes that the kernels do not take, results
that are written to, masks that follow the model's seed, state and replays."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def small(d=192, heads=4, dropout=0.0, seed=0, layers=2):
    from coo_spmm_sparse_gb300.decoder import DecoderConfig, SparseDecoder
    return SparseDecoder(DecoderConfig(vocab=128, ctx=64, d=d, heads=heads, layers=layers, mlp=2 * d, sparsity=80.0,
                                       std=0.1, dropout=dropout, seed=seed))


def tokens(n=2, length=64, seed=0):
    return torch.randint(0, 128, (n, length), generator=torch.Generator().manual_seed(seed)).cuda()


def test_heads_of_more_than_128_columns():
    """A chain of some 20 fp32 operations against the same in 64 bits: 1e-3 of the largest."""
    from test_gpu_attention_decoder import plain
    from coo_spmm_sparse_gb300.decoder import Trainer
    from coo_spmm_sparse_gb300.finetune import AdaptedDecoder, FineTuner, sequences
    model, idx = small(d=512, heads=2), tokens()
    got, want = model(idx).detach(), plain(model, idx).detach()
    assert float((got.double() - want).abs().max()) <= 1e-3 * float(want.abs().max())
    assert torch.isfinite(Trainer(model, prune_every=0).step(idx))
    loss, _ = FineTuner(AdaptedDecoder(model, adapters=2, rank=4)).step(idx, sequences(2, 64, [0, 1]))
    assert torch.isfinite(loss)
    with pytest.raises(ValueError, match="at most 128"):
        small(d=512, heads=2, dropout=0.1)(idx)


@pytest.mark.parametrize("ragged", [False, True])
def test_packed_attention_can_be_written_to(ragged):
    """The result is no view: it may be written to in grad mode.  As for any function that keeps its
    result for the gradient, a backward pass through the old value then raises."""
    import coo_spmm_sparse_gb300 as sn
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (90,) if ragged else (2, 45)
    offsets = torch.tensor([0, 30, 90], dtype=torch.int32, device="cuda") if ragged else None
    qkv = torch.randn(*shape, 8 * 32, generator=g, device="cuda", requires_grad=True)
    out = sn.snack_packed_attention(qkv, 4, 2, offsets=offsets)
    assert out.shape == (*shape, 128) and out._base is None
    keep = out.detach().clone()
    out += 1.0
    assert torch.equal(out.detach(), keep + 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    with torch.no_grad():
        again = sn.snack_packed_attention(qkv, 4, 2, offsets=offsets)
    again.mul_(2.0)
    assert torch.equal(again, keep * 2.0)
    empty = sn.snack_packed_attention(qkv[:0].detach().requires_grad_(), 4, 2,
                                      offsets=offsets[:1] if ragged else None)
    assert empty.shape == (0, *shape[1:], 128)
    empty.sum().backward()
