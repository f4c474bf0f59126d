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


def test_masks_are_part_of_the_models_state():
    a, idx = small(dropout=0.2), tokens()
    first = [a(idx).detach() for _ in range(3)]
    assert a.calls == 3 and not torch.equal(first[0], first[1])
    b = small(dropout=0.2)
    b.load_state_dict(a.state_dict())
    assert b.calls == 3
    assert torch.equal(a(idx), b(idx))
    for n in range(3):
        assert torch.equal(b(idx, call=n), first[n])
    assert b.calls == 4
    b.eval()
    b(idx)
    assert b.calls == 4
    plain = small()
    assert not [k for k in plain.state_dict() if "_calls" in k or "_places" in k]
    older = {k: v for k, v in a.state_dict().items() if k != "_calls"}
    small(dropout=0.2).load_state_dict(older)
    plain.load_state_dict(older)
    plain.load_state_dict(a.state_dict())


def test_masks_follow_the_models_seed():
    from coo_spmm_sparse_gb300.decoder import DecoderConfig, SparseDecoder
    import attention_ref
    idx = tokens()
    base = dict(vocab=128, ctx=64, d=192, heads=4, layers=1, mlp=384, sparsity=80.0, std=0.1, dropout=0.2)
    a = SparseDecoder(DecoderConfig(**base))
    others = [SparseDecoder(DecoderConfig(**base, mask_seed=m)) for m in (0, 1, 2)]
    got = [m(idx) for m in (a, *others)]
    assert torch.equal(got[0], got[1])
    assert not torch.equal(got[1], got[2]) and not torch.equal(got[2], got[3])
    assert [int(s) for s in others[2].mask_seeds()[1][:2]] == [2 * 2 ** 40 + 4096, 2 * 2 ** 40 + 4097]
    # the embeddings' mask is that of the documented seed
    x = torch.ones(300, device="cuda")
    import coo_spmm_sparse_gb300 as sn
    M = attention_ref.mask_of(2 ** 40 + 4096 * 5, torch.zeros(1, dtype=torch.long, device="cuda"), 300, 0.2)
    assert torch.equal(sn.snack_dropout_forward(x, 0.2, others[1].mask_seeds(call=5)[1][0]) != 0, M.flatten() != 0)


def test_a_captured_call_draws_new_masks_at_every_replay():
    model, idx = small(dropout=0.2), tokens()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.no_grad(), torch.cuda.stream(side):
        model(idx)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        logits = model(idx)
    start = model.calls
    for n in range(3):
        graph.replay()
        got = logits.clone()
        with torch.no_grad():
            assert torch.equal(got, model(idx, call=start + n))
    assert model.calls == start + 3


def test_a_call_that_is_made_again_draws_its_own_masks():
    from torch.utils.checkpoint import checkpoint
    model, idx = small(dropout=0.2), tokens()
    model(idx, call=7).sum().backward()
    want = {n: p.grad.clone() for n, p in model.named_parameters()}
    model.zero_grad()
    checkpoint(lambda i: model(i, call=7), idx, use_reentrant=False).sum().backward()
    for n, p in model.named_parameters():
        assert torch.allclose(p.grad, want[n], rtol=1e-4, atol=1e-5 * float(want[n].abs().max())), n
    with pytest.raises(RuntimeError, match="call=n"):
        checkpoint(lambda i: model(i), idx, use_reentrant=False).sum().backward()


def test_adapted_decoder_drops_what_its_base_drops():
    """New adapters add nothing: the logits of a call are the base's of the same call, in training
    mode with its masks (two orders of 32-bit sums: 1e-4 of the largest), outside it without."""
    from coo_spmm_sparse_gb300.finetune import AdaptedDecoder, FineTuner, sequences
    base, idx = small(dropout=0.3), tokens()
    model = AdaptedDecoder(base, adapters=2, rank=4)
    requests = sequences(2, 64, [0, 1])
    with torch.no_grad():
        want, got = base(idx, call=3), model(idx, requests, call=3)
        assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max())
        other = model(idx, requests, call=4)
        assert float((other - want).abs().max()) > 1e-2 * float(want.abs().max())
        model.eval()
        want = base(idx)
        assert float((model(idx, requests) - want).abs().max()) <= 1e-4 * float(want.abs().max())
        model.train()
    assert base.calls == 0
    loss, _ = FineTuner(model).step(idx, requests)
    assert torch.isfinite(loss) and base.calls == 1


def test_the_decoders_attention_within_its_own_bounds():
    """What every block of a training call passes to the attention and gets back, forward and backward,
    held to the operator's own bounds (products in one tf32 part would miss them)."""
    import attention_ref
    from coo_spmm_sparse_gb300 import decoder
    model, idx = small(d=256, heads=4), tokens(n=12)
    calls, plain = [], decoder.attend

    def attend(qkv, heads, dropout=0.0, seed=0):
        a = plain(qkv, heads, dropout, seed)
        qkv.retain_grad()
        a.retain_grad()
        calls.append((qkv, a))
        return a

    decoder.attend = attend
    try:
        (model(idx) * torch.randn(12, 64, 128, device="cuda")).sum().backward()
    finally:
        decoder.attend = plain
    assert len(calls) == 2
    for qkv, a in calls:
        q, k, v = (t.unflatten(-1, (4, 64)) for t in qkv.detach().split(256, -1))
        want = attention_ref.attention(q, k, v, dout=a.grad.unflatten(-1, (4, 64)))
        grads = qkv.grad.unflatten(-1, (3, 4, 64)).unbind(-3)
        attention_ref.assert_within(dict(zip(("out", "dq", "dk", "dv"), (a.detach().unflatten(-1, (4, 64)), *grads))),
                                    want)
        rough = [t.to(torch.float32).view(torch.int32).bitwise_and(-8192).view(torch.float32) for t in (q, k, v)]
        other = attention_ref.attention(*rough)["out"][0]  # operands cut to tf32 are outside them
        assert bool(((other - want["out"][0]).abs() > want["out"][1]).any())
