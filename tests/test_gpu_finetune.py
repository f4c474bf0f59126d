"""Adapters, block norms and clipping together: the fine-tuned sparse decoder."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def small():
    from coo_spmm_sparse_gb300.decoder import DecoderConfig, SparseDecoder
    cfg = DecoderConfig(vocab=512, ctx=64, d=192, heads=4, layers=2, mlp=384, sparsity=90.0, std=0.1)
    return cfg, SparseDecoder(cfg)


def test_new_adapters_leave_the_decoder_as_it_is():
    from coo_spmm_sparse_gb300.finetune import AdaptedDecoder, sequences
    cfg, base = small()
    idx = torch.randint(0, cfg.vocab, (3, cfg.ctx), device="cuda")
    with torch.no_grad():
        want = base(idx)
        model = AdaptedDecoder(base, adapters=3, rank=4)
        got = model(idx, sequences(3, cfg.ctx, [0, -1, 2]))
    # the same layer norms with their sums in another order, through two blocks
    assert torch.allclose(got, want, rtol=1e-4, atol=1e-4 * float(want.abs().max()))


def test_fine_tuning_changes_only_the_adapters_that_were_used():
    from coo_spmm_sparse_gb300.finetune import AdaptedDecoder, FineTuner, sequences
    cfg, base = small()
    frozen = {k: v.clone() for k, v in base.state_dict().items()}
    model = AdaptedDecoder(base, adapters=3, rank=4, sandwich=True)
    tuner = FineTuner(model, lr=0.5, max_norm=0.5)
    g = torch.Generator().manual_seed(1)
    idx = torch.randint(0, cfg.vocab, (2, cfg.ctx), generator=g).cuda()
    requests = sequences(2, cfg.ctx, [0, 2])
    losses, norms = [], []
    for _ in range(30):
        loss, norm = tuner.step(idx, requests)
        losses.append(float(loss))
        norms.append(float(norm))
    assert all(n == n and n > 0 for n in norms)
    assert losses[-1] < losses[0] - 0.05, losses
    for k, v in base.state_dict().items():
        assert torch.equal(v, frozen[k]), k
    for b in model.blocks:
        for ad in b.adapters:
            assert not ad.B[1].any()  # no request named adapter 1
            assert ad.B[0].any() and ad.B[2].any()


def test_one_batch_serves_each_request_its_own_adapter():
    from coo_spmm_sparse_gb300.finetune import AdaptedDecoder, sequences
    cfg, base = small()
    model = AdaptedDecoder(base, adapters=2, rank=4)
    with torch.no_grad():
        for b in model.blocks:
            for ad in b.adapters:
                ad.B.normal_(0, 0.1)
        idx = torch.randint(0, cfg.vocab, (1, cfg.ctx), device="cuda").expand(4, -1).contiguous()
        together = model(idx, sequences(4, cfg.ctx, [1, -1, 0, 1]))
        for row, n in enumerate([1, -1, 0, 1]):
            alone = model(idx[:1], sequences(1, cfg.ctx, [n]))[0]
            assert torch.allclose(together[row], alone, rtol=1e-4, atol=1e-4 * float(alone.abs().max()))
    assert float((together[0] - together[2]).abs().max()) > 1e-2


def test_clipped_gradients_have_the_norm_asked_for():
    from coo_spmm_sparse_gb300 import snack_clip_grad_norm, snack_grad_norm
    from coo_spmm_sparse_gb300.finetune import AdaptedDecoder, sequences
    cfg, base = small()
    model = AdaptedDecoder(base, adapters=1, rank=4)
    idx = torch.randint(0, cfg.vocab, (1, cfg.ctx), device="cuda")
    model.loss(idx, sequences(1, cfg.ctx, [0])).backward()
    grads = [p.grad for p in model.trained() if p.grad is not None]
    want = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
    got = snack_clip_grad_norm(grads, 0.1 * float(want))
    assert abs(float(got) - float(want)) <= 1e-5 * float(want)
    assert abs(float(snack_grad_norm(grads)) - 0.1 * float(want)) <= 1e-4 * float(want)
