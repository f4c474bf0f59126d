"""Fine-tuning the sparse decoder by low-rank adapters, and serving several of
them at once: the sparse projections stay as they are and are shared, every
request brings its own adapter.

``AdaptedDecoder`` holds a ``SparseDecoder`` whose parameters are frozen and,
beside each of its 48 sparse projections, ``SnackAdapters`` for a number of
adapters.  Its blocks run through ``snack_residual_norm``: the add of a
block's output and the layer norm that follows are one call, optionally with
a norm of the output itself and a learned gate per channel.  With new
adapters (B = 0), gates of 1 and no output norm it computes what the decoder
it wraps computes.

``FineTuner`` trains the adapters and gates: plain SGD on gradients clipped
to a global norm (``snack_clip_grad_norm`` over all of them).

    python -m coo_spmm_sparse_gb300.finetune            # a short run on random tokens
"""

from __future__ import annotations

import torch
import torch.nn.functional as F

from . import SnackAdapters, SnackResidualNorm, snack_clip_grad_norm, snack_residual_norm
from .decoder import DecoderConfig, SparseDecoder


class AdaptedBlock(torch.nn.Module):
    """A block of the decoder with adapters beside its projections."""

    def __init__(self, block, d: int, mlp: int, adapters: int, rank: int, alpha: float,
                 sandwich: bool, seed: int):
        super().__init__()
        self.block = block
        shapes = [(d, 3 * d), (d, d), (d, mlp), (mlp, d)]
        self.adapters = torch.nn.ModuleList(
            SnackAdapters(adapters, i, o, rank, alpha, seed=seed + k)
            for k, (i, o) in enumerate(shapes))
        # after the attention and after the MLP; the norms that follow are the decoder's own
        self.joins = torch.nn.ModuleList(
            SnackResidualNorm(d, post=sandwich, next=False, gate="channel") for _ in range(2))

    def project(self, k: int, lin, x, requests):
        return self.adapters[k](x, lin(x), *requests)

    def attention(self, h, requests):
        b = self.block
        B, T, d = h.shape
        q, k, v = self.project(0, b.c_attn, h, requests).split(d, dim=2)
        q, k, v = (t.view(B, T, b.heads, d // b.heads).transpose(1, 2) for t in (q, k, v))
        a = F.scaled_dot_product_attention(q, k, v, is_causal=True)
        return self.project(1, b.attn_c_proj, a.transpose(1, 2).reshape(B, T, d), requests)

    def mlp(self, h, requests):
        b = self.block
        return self.project(3, b.mlp_c_proj,
                            F.gelu(self.project(2, b.c_fc, h, requests), approximate="tanh"),
                            requests)


def _join(norm: SnackResidualNorm, x, y, following: torch.nn.LayerNorm):
    """(r, h): y joined to the residual x, and the layer norm that the next block reads."""
    return snack_residual_norm(x, y, gate=norm.gate, post_weight=norm.post_weight,
                               post_bias=norm.post_bias, next_weight=following.weight,
                               next_bias=following.bias, eps=following.eps,
                               post_norm=norm.opts["post_norm"])


class AdaptedDecoder(torch.nn.Module):
    """A frozen sparse decoder with adapters.  ``requests`` of a call is
    (offsets, adapter): request i owns the tokens offsets[i] .. offsets[i+1]-1
    of the flattened batch and uses adapter[i] (-1: the decoder as it is)."""

    def __init__(self, base: SparseDecoder, adapters: int = 1, rank: int = 8,
                 alpha: float | None = None, sandwich: bool = False, seed: int = 0):
        super().__init__()
        self.base = base
        for p in base.parameters():
            p.requires_grad_(False)
        cfg = base.cfg
        self.blocks = torch.nn.ModuleList(
            AdaptedBlock(b, cfg.d, cfg.mlp, adapters, rank, rank if alpha is None else alpha,
                         sandwich, seed + 10 * i) for i, b in enumerate(base.blocks))

    def trained(self):
        """The parameters that fine-tuning changes."""
        return [p for p in self.parameters() if p.requires_grad]

    def forward(self, idx: torch.Tensor, requests) -> torch.Tensor:
        base = self.base
        pos = torch.arange(idx.shape[1], device=idx.device)
        x = base.wte(idx) + base.wpe(pos)
        first = base.blocks[0].ln_1
        x, h = snack_residual_norm(x, next_weight=first.weight, next_bias=first.bias,
                                   eps=first.eps)
        for i, b in enumerate(self.blocks):
            x, h = _join(b.joins[0], x, b.attention(h, requests), b.block.ln_2)
            after = base.blocks[i + 1].ln_1 if i + 1 < len(self.blocks) else base.ln_f
            x, h = _join(b.joins[1], x, b.mlp(h, requests), after)
        return F.linear(h, base.wte.weight)

    def loss(self, idx: torch.Tensor, requests) -> torch.Tensor:
        """Next-token cross-entropy of a [B][T] token batch."""
        logits = self.forward(idx, requests)
        return F.cross_entropy(logits[:, :-1].reshape(-1, logits.shape[-1]),
                               idx[:, 1:].reshape(-1))


class FineTuner:
    """SGD on the adapters and gates, their gradients clipped to a global norm."""

    def __init__(self, model: AdaptedDecoder, lr: float = 0.1, max_norm: float = 1.0):
        self.model, self.max_norm = model, max_norm
        self.params = model.trained()
        self.opt = torch.optim.SGD(self.params, lr=lr)

    def step(self, idx: torch.Tensor, requests):
        """One step; returns (loss, gradient norm before clipping), on the device."""
        self.opt.zero_grad(set_to_none=True)
        loss = self.model.loss(idx, requests)
        loss.backward()
        norm = snack_clip_grad_norm([p.grad for p in self.params if p.grad is not None],
                                    self.max_norm)
        self.opt.step()
        return loss.detach(), norm


def sequences(batch: int, ctx: int, adapter, device="cuda"):
    """(offsets, adapter) of `batch` sequences of `ctx` tokens, one request each."""
    offsets = torch.arange(batch + 1, dtype=torch.int32, device=device) * ctx
    return offsets, torch.as_tensor(adapter, dtype=torch.int32, device=device)


def main():
    cfg = DecoderConfig()
    model = AdaptedDecoder(SparseDecoder(cfg), adapters=2, rank=8, sandwich=False)
    tuner = FineTuner(model)
    g = torch.Generator().manual_seed(0)
    idx = torch.randint(0, cfg.vocab, (2, cfg.ctx), generator=g).cuda()
    requests = sequences(2, cfg.ctx, [0, 1])
    for step in range(20):
        loss, norm = tuner.step(idx, requests)
        if step % 5 == 0 or step == 19:
            print(f"step {step}: loss {float(loss):.4f}, gradient norm {float(norm):.4f}")
    with torch.no_grad():  # one batch: a sequence with each adapter, one without
        three = torch.cat([idx[:1], idx[:1], idx[:1]])
        logits = model(three, sequences(3, cfg.ctx, [0, 1, -1]))
    print("logits of one prompt under adapter 0, 1 and none differ by",
          [round(float((logits[a] - logits[b]).abs().max()), 4) for a, b in ((0, 1), (0, 2))])


if __name__ == "__main__":
    main()
