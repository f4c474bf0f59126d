"""GPT-2-small-shaped decoder whose attention and MLP projections are SNACK
sparse layers: the training harness of the paper's GPT-2 dynamic-sparse runs
("Beyond Masked Sparsity: SNACK Enables Truly Sparse Neural Networks on
GPU", §5 Tables 4-5; Appendix G "Sparsity schedule and DST"), on random
tokens instead of WikiText-103.

Every block's four projections (c_attn 768->2304, attention c_proj
768->768, c_fc 768->3072, MLP c_proj 3072->768) are ``SnackLinear`` layers
at the given sparsity: their forward and backward run in the library's
kernels, and so does the causal attention between them
(``snack_packed_attention`` on c_attn's output; heads of more than 128
columns, which it does not take, attend through PyTorch, without dropout).
Token and position embeddings, layer norms, GELU and the tied LM head stay dense PyTorch: the
paper makes only the Linear projections sparse.

``dropout`` (0 by default) is GPT-2's: of the embeddings, of the attention's
probabilities and of a block's outputs before they join the residual stream,
while the model is in training mode.  Call n of the model draws its masks
from seeds 2^40 * mask_seed + 4096 * n + place (place 0: the embeddings;
4 i + 1 .. 4 i + 3: block i), on the device.  n counts the calls in a buffer
that is part of the state of a model with dropout, and of a captured step; a
call that is made again (activation checkpointing) has to name its n.

The training step is plain SGD on every parameter (the sparse values are
updated in place through their Parameter views) and, every
``prune_every`` steps, a magnitude-prune / uniform-regrow of each sparse
layer (Appendix G) with a per-layer seed derived from the step.
"""

from __future__ import annotations

import math
from dataclasses import dataclass

import torch
import torch.nn.functional as F

from . import SnackLinear, snack_dropout, snack_packed_attention


def nnz_for(out: int, inp: int, sparsity_pct: float) -> int:
    """Stored entries of an out x in layer: (1 - sparsity) * out * in,
    rounded half up (256x256 at 90 % -> 6554)."""
    x = (100.0 - sparsity_pct) * out * inp
    return int(math.floor(x / 100.0 + 0.5))


@dataclass
class DecoderConfig:
    vocab: int = 50257
    ctx: int = 256
    d: int = 768
    heads: int = 12
    layers: int = 12
    mlp: int = 3072
    sparsity: float = 99.0
    std: float = 0.02
    seed: int = 0
    dropout: float = 0.0
    mask_seed: int | None = None  # of dropout's masks, below 2^23; None: seed.  Ranks take unlike ones


class Block(torch.nn.Module):
    def __init__(self, cfg: DecoderConfig, index: int):
        super().__init__()
        d, m = cfg.d, cfg.mlp
        self.heads = cfg.heads
        self.ln_1 = torch.nn.LayerNorm(d)
        self.ln_2 = torch.nn.LayerNorm(d)

        def sparse(j, inp, out):
            return SnackLinear(inp, out, nnz_for(out, inp, cfg.sparsity),
                               seed=cfg.seed + 1000 * index + j, std=cfg.std)

        self.c_attn = sparse(0, d, 3 * d)
        self.attn_c_proj = sparse(1, d, d)
        self.c_fc = sparse(2, d, m)
        self.mlp_c_proj = sparse(3, m, d)

    def sparse_layers(self):
        return [self.c_attn, self.attn_c_proj, self.c_fc, self.mlp_c_proj]

    def forward(self, x: torch.Tensor, dropout: float = 0.0, seeds=(0, 0, 0)) -> torch.Tensor:
        a = attend(self.c_attn(self.ln_1(x)), self.heads, dropout, seeds[0])
        x = join(x, self.attn_c_proj(a), dropout, seeds[1])
        return join(x, self.mlp_c_proj(F.gelu(self.c_fc(self.ln_2(x)), approximate="tanh")),
                    dropout, seeds[2])


def attend(qkv: torch.Tensor, heads: int, dropout: float = 0.0, seed=0) -> torch.Tensor:
    """Causal self-attention of a projection's output [B][T][3 * d]."""
    B, T, width = qkv.shape
    if width // (3 * heads) <= 128:
        return snack_packed_attention(qkv, heads, dropout=dropout, seed=seed)
    if dropout:
        raise ValueError("dropout takes heads of at most 128 columns")
    q, k, v = (t.unflatten(-1, (heads, -1)).transpose(1, 2) for t in qkv.split(width // 3, dim=-1))
    return F.scaled_dot_product_attention(q, k, v, is_causal=True).transpose(1, 2).flatten(-2)


def join(x: torch.Tensor, y: torch.Tensor, dropout: float, seed) -> torch.Tensor:
    """x + y, with dropout of y."""
    return snack_dropout(y, dropout, seed, residual=x) if dropout else x + y


class SparseDecoder(torch.nn.Module):
    """GPT-2-small-shaped decoder with SNACK sparse projections."""

    def __init__(self, cfg: DecoderConfig = DecoderConfig(), device=None):
        super().__init__()
        self.cfg = cfg
        dev = device or torch.device("cuda", torch.cuda.current_device())
        g = torch.Generator(device="cpu").manual_seed(cfg.seed)
        self.wte = torch.nn.Embedding(cfg.vocab, cfg.d, device=dev)
        self.wpe = torch.nn.Embedding(cfg.ctx, cfg.d, device=dev)
        with torch.no_grad():
            self.wte.weight.copy_(torch.randn(cfg.vocab, cfg.d, generator=g) * cfg.std)
            self.wpe.weight.copy_(torch.randn(cfg.ctx, cfg.d, generator=g) * 0.01)
        self.blocks = torch.nn.ModuleList(Block(cfg, i) for i in range(cfg.layers))
        self.ln_f = torch.nn.LayerNorm(cfg.d, device=dev)
        mask_seed = cfg.seed if cfg.mask_seed is None else cfg.mask_seed
        self.register_buffer("_calls", torch.zeros((), dtype=torch.long), persistent=cfg.dropout > 0)
        self.register_buffer("_places", torch.arange(4 * cfg.layers + 1) + (mask_seed % 2 ** 23 << 40),
                             persistent=False)
        self.to(dev)

    @property
    def calls(self) -> int:
        """Calls with dropout so far (read from the device)."""
        return int(self._calls)

    @calls.setter
    def calls(self, n: int):
        self._calls.fill_(n)

    def _load_from_state_dict(self, state_dict, prefix, *args):
        if self.cfg.dropout:  # a state of a model without dropout, or from before the calls were part of it
            state_dict.setdefault(prefix + "_calls", self._calls)
        else:
            state_dict.pop(prefix + "_calls", None)
        super()._load_from_state_dict(state_dict, prefix, *args)

    def mask_seeds(self, call: int | None = None):
        """(dropout, seeds of the places) of a call: the next one, which is counted, or number `call`."""
        p = self.cfg.dropout if self.training else 0.0
        if not p:
            return 0.0, [0] * (4 * self.cfg.layers + 1)
        if 4 * self.cfg.layers >= 4096:
            raise ValueError("dropout takes at most 1023 blocks")
        if call is not None:
            return p, (self._places + 4096 * call).unbind()
        if torch._C._current_graph_task_id() != -1:
            raise RuntimeError("a call inside a backward pass (activation checkpointing) would draw other masks "
                               "than the one it repeats: give both the call's number, model(idx, call=n)")
        seeds = torch.add(self._places, self._calls, alpha=4096).unbind()
        self._calls.add_(1)
        return p, seeds

    def sparse_layers(self):
        return [lin for b in self.blocks for lin in b.sparse_layers()]

    def forward(self, idx: torch.Tensor, call: int | None = None) -> torch.Tensor:
        B, T = idx.shape
        pos = torch.arange(T, device=idx.device)
        x = self.wte(idx) + self.wpe(pos)
        p, seeds = self.mask_seeds(call)
        if p:
            x = snack_dropout(x, p, seeds[0])
        for i, b in enumerate(self.blocks):
            x = b(x, p, seeds[4 * i + 1: 4 * i + 4])
        return F.linear(self.ln_f(x), self.wte.weight)  # tied LM head

    def loss(self, idx: torch.Tensor, call: int | None = None) -> torch.Tensor:
        """Next-token cross-entropy of a [B][T] token batch."""
        logits = self.forward(idx, call)
        return F.cross_entropy(logits[:, :-1].reshape(-1, logits.shape[-1]),
                               idx[:, 1:].reshape(-1))

    @torch.no_grad()
    def prune_regrow(self, frac: float, step: int):
        """Magnitude-prune / uniform-regrow every sparse layer (Appendix G);
        layer i uses seed 7919 * step + i.  Returns [(pruned, trials)]."""
        return [lin.prune_regrow(frac, 7919 * step + i) for i, lin in
                enumerate(self.sparse_layers())]


class Trainer:
    """Plain SGD (no momentum) on every parameter, with prune/regrow of the
    sparse layers every ``prune_every`` steps."""

    def __init__(self, model: SparseDecoder, lr: float = 1e-2, prune_frac: float = 0.30,
                 prune_every: int = 100):
        self.model = model
        self.opt = torch.optim.SGD(model.parameters(), lr=lr, momentum=0.0)
        self.prune_frac, self.prune_every = prune_frac, prune_every
        self.step_no = 0

    def step(self, idx: torch.Tensor) -> torch.Tensor:
        """One training step on a token batch; returns the loss (on device)."""
        self.opt.zero_grad(set_to_none=True)
        loss = self.model.loss(idx)
        loss.backward()
        self.opt.step()
        self.step_no += 1
        if self.prune_every and self.step_no % self.prune_every == 0:
            self.model.prune_regrow(self.prune_frac, self.step_no)
        return loss.detach()
