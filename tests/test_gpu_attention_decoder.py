"""Attention and dropout as the decoder uses them: one block against a plain 64-bit
evaluation, training with dropout, adapters and clipping around both."""

import pytest
import torch
import torch.nn.functional as F

import attention_ref

pytestmark = pytest.mark.gpu


def small(dropout=0.0):
    from coo_spmm_sparse_gb300.decoder import DecoderConfig, SparseDecoder
    return SparseDecoder(DecoderConfig(vocab=512, ctx=96, d=192, heads=4, layers=2, mlp=384, sparsity=80.0,
                                       std=0.1, dropout=dropout))


def dense_weight(lin):
    row, col, val = lin.export()
    W = torch.zeros(lin.out_features, lin.in_features, dtype=torch.float64)
    W[torch.as_tensor(row).long(), torch.as_tensor(col).long()] = torch.as_tensor(val).double()
    return W.cuda()


def plain(model, idx, p=0.0, call=0):
    """Logits in 64 bits from the definitions, masks from the documented seeds."""
    f = torch.float64
    cfg, d = model.cfg, model.cfg.d
    B, T = idx.shape
    seed = 4096 * call

    def drop(y, s):
        if not p:
            return y
        M = attention_ref.mask_of(s, torch.zeros(1, dtype=torch.long, device="cuda"), y.numel(), p)
        return y * M.view(y.shape)

    def lin(m, x):
        return x @ dense_weight(m).T + m.bias.to(f)

    def norm(m, x):
        return F.layer_norm(x, (d,), m.weight.to(f), m.bias.to(f), m.eps)

    x = drop(model.wte.weight.to(f)[idx] + model.wpe.weight.to(f)[:T], seed)
    for i, b in enumerate(model.blocks):
        s = seed + 4 * i + 1
        q, k, v = (t.view(B, T, cfg.heads, -1).transpose(1, 2) for t in lin(b.c_attn, norm(b.ln_1, x)).split(d, -1))
        scores = q @ k.mT / (d // cfg.heads) ** 0.5
        P = torch.softmax(scores.masked_fill(~torch.ones(T, T, dtype=torch.bool, device="cuda").tril(), -torch.inf), -1)
        if p:
            rows = torch.arange(B * T, device="cuda").view(B, 1, T) * cfg.heads
            P = P * attention_ref.mask_of(s, (rows + torch.arange(cfg.heads, device="cuda")[:, None]) << 30, T, p)
        a = (P @ v).transpose(1, 2).reshape(B, T, d)
        x = x + drop(lin(b.attn_c_proj, a), s + 1)
        h = F.gelu(lin(b.c_fc, norm(b.ln_2, x)), approximate="tanh")
        x = x + drop(lin(b.mlp_c_proj, h), s + 2)
    return norm(model.ln_f, x) @ model.wte.weight.to(f).T


@pytest.mark.parametrize("dropout", [0.0, 0.1])
def test_decoder_with_attention_and_dropout(dropout):
    """Logits and the embedding's gradient: a chain of some 20 fp32 operations, each with the
    1e-5 of its terms that its own test allows; 1e-3 of the largest covers their sum."""
    model = small(dropout)
    idx = torch.randint(0, 512, (2, 96), generator=torch.Generator().manual_seed(0)).cuda()
    for call in range(2):
        want = plain(model, idx, dropout, call)
        got = model(idx)
        assert float((got.double() - want).abs().max()) <= 1e-3 * float(want.abs().max())
    model.zero_grad()
    model.eval()
    a = model(idx)
    assert torch.equal(a, model(idx))  # no masks outside training
    model.train()
    w = torch.randn_like(a)
    call = model.calls
    (model(idx) * w).sum().backward()
    leaf = model.wpe.weight.detach().double().requires_grad_()

    class View:  # the same model with its position embeddings as a 64-bit leaf
        cfg, wte, blocks, ln_f = model.cfg, model.wte, model.blocks, model.ln_f
        wpe = type("W", (), {"weight": leaf})

    (plain(View, idx, dropout, call) * w).sum().backward()
    assert float((model.wpe.weight.grad.double() - leaf.grad).abs().max()) <= 1e-3 * float(leaf.grad.abs().max())


def test_training_step_with_dropout_adapters_and_clipping():
    """The operators together, as a fine-tuning step uses them: adapters beside the projections,
    norms that join, packed attention, clipping; then the decoder's own step with dropout."""
    from coo_spmm_sparse_gb300.decoder import Trainer
    from coo_spmm_sparse_gb300.finetune import AdaptedDecoder, FineTuner, sequences
    base = small(0.1)
    idx = torch.randint(0, 512, (2, 96), generator=torch.Generator().manual_seed(1)).cuda()
    loss = Trainer(base, prune_every=0).step(idx)
    assert torch.isfinite(loss) and base.calls == 1
    for p in base.parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all()
    tuner = FineTuner(AdaptedDecoder(base, adapters=2, rank=4))
    loss, norm = tuner.step(idx, sequences(2, 96, [0, 1]))
    assert torch.isfinite(loss) and float(norm) > 0
