"""Cases that time the attention of the decoder around its sparse projections,
forward and backward, and the dropout that its training uses.

Attention of query head h over the keys of head h // (heads / key heads), for
query i of a sequence with nq queries and nk keys (causal: key j is seen where
j <= i + nk - nq):

    P[i, j] = exp(scale * q_i . k_j) / sum over the seen keys (a row that sees none is zero)
    out_i = sum_j M[i, j] * P[i, j] * v_j

Dropout: y = residual + M * x.  Element e of a tensor (or key j of a
probability row r = token * heads + head, as e = r * 2^32 + j) takes bits
16 * (e mod 4) and up of the SplitMix64 draw number e / 4 of the seed; it is
kept where these 16 bits are at least T = round(65536 p), M is then
65536 / (65536 - T), else 0.

``run`` computes a case in plain torch (32-bit arithmetic, one rounding at the
end), or, with ``own`` set, through the package's entry points.  ``exact``
evaluates the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _attn(name, layout, seqs, q, k, heads, key_heads, d, dtype, causal, dropout, train):
    """layout "dense": seqs sequences of q queries and k keys; "padded": of at most q tokens;
    "cache": q new tokens each over caches with room for k keys; "ragged": q and k tokens in all."""
    return {"name": name, "op": "attention", "layout": layout, "seqs": seqs, "q": q, "k": k,
            "heads": heads, "key_heads": key_heads, "d": d, "dtype": dtype, "causal": causal,
            "dropout": dropout, "train": train}


def _drop(name, rows, d, stream, branch, residual, p, train):
    return {"name": name, "op": "dropout", "rows": rows, "d": d, "stream": stream,
            "branch": branch, "residual": residual, "p": p, "train": train}


def listed():
    return [
        # One decoded token of the GPT-2-small-shaped decoder at the end of its context: latency alone.
        _attn("attn_token", "cache", 1, 1, 256, 12, 12, 64, "f32", True, 0.0, False),
        # Decoding a batch of requests over long caches of unlike fill: the caches' bytes are the work.
        _attn("attn_caches", "cache", 16, 1, 32768, 32, 8, 128, "bf16", True, 0.0, False),
        # Prompts of ragged lengths packed end to end, at a head size no power of two.
        _attn("attn_prompts", "ragged", 13, 6001, 6001, 16, 4, 80, "f16", True, 0.0, False),
        # One long prompt.
        _attn("attn_prefill", "dense", 1, 16384, 16384, 16, 2, 128, "bf16", True, 0.0, False),
        # The decoder's training step on its context of 256 tokens, with GPT-2's dropout.
        _attn("attn_context_train", "dense", 1, 256, 256, 12, 12, 64, "f32", True, 0.1, True),
        # Training on a padded batch of sequences in 32 bits.
        _attn("attn_padded_train", "padded", 8, 1023, 1023, 12, 12, 64, "f32", True, 0.0, True),
        # Fine-tuning on documents packed end to end, grouped heads.
        _attn("attn_packed_train", "ragged", 9, 8191, 8191, 24, 8, 64, "bf16", True, 0.0, True),
        # Pre-training of a wide model on long sequences.
        _attn("attn_long_train", "dense", 1, 8192, 8192, 32, 8, 128, "bf16", True, 0.0, True),
        # The add of a block's output to the residual stream in the decoder's training step.
        _drop("dropout_context_train", 256, 768, "f32", "f32", True, 0.1, True),
        # The same at an odd width, a 16-bit branch on a 32-bit residual stream.
        _drop("dropout_odd_train", 4095, 1001, "f32", "bf16", True, 0.1, True),
        # Pre-training of a wide model.
        _drop("dropout_wide_train", 16384, 4096, "bf16", "bf16", True, 0.1, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.25:
        stream, branch = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                     ("f32", "bf16"), ("f32", "f16")])
        d = _log_int(rng, 64, 8192)
        rows = _log_int(rng, 1, max(2, min(16384, 16384 * 4096 // d)))
        c = _drop("", rows, d, stream, branch, rng.random() < 0.7,
                  rng.choice([0.05, 0.1, 0.1, 0.2, 0.5]), rng.random() < 0.7)
        del c["name"]
        return c
    train = rng.random() < 0.5
    layout = rng.choice(["dense", "padded", "ragged"] if train else ["dense", "cache", "cache", "ragged"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    key_heads, group = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([1, 1, 2, 3, 4, 8])
    while key_heads * group > 32:
        group -= 1
    d = rng.choice([64, 64, 64, 128, 128, 128, 32, 48, 72, 80, 96, 100, 65])
    dropout = rng.choice([0.0, 0.0, 0.1, 0.2]) if train else 0.0
    seqs = _log_int(rng, 1, 16)
    if layout == "cache":
        k = _log_int(rng, 64, 32768)
        q = rng.choice([1, 1, 1, 2, 5, 8, 64])
    else:
        q = _log_int(rng, 1, 8192)
        # a sixth of the cases attends to another sequence
        k = _log_int(rng, 1, 8192) if layout != "padded" and rng.random() < 1 / 6 else q
    # no dearer than the largest listed case of the direction; a seventh of that in 32 bits or with dropout
    most = (16 if train else 4) * 8192 * 8192 * 16 * 64 // (7 if dtype == "f32" or dropout else 1)
    while seqs > 1 and seqs * q * k * key_heads * group * d > most and layout != "ragged":
        seqs //= 2
    while q * k * seqs * key_heads * group * d > most and q > 1 and layout != "ragged":
        q, k = q // 2, (k + 1) // 2
    while layout == "ragged" and q * k * key_heads * group * d > most:
        q, k = (q + 1) // 2, (k + 1) // 2
    c = _attn("", layout, seqs, q, k, key_heads * group, key_heads, d, dtype,
              rng.random() < 0.8, dropout, train)
    del c["name"]
    return c


def _parts(total, n, salt):
    """n lengths, log-normal, that sum to total; now and then an empty one."""
    g = torch.Generator().manual_seed(1000 * n + salt)
    w = torch.exp(torch.randn(n, generator=g, dtype=torch.float64) * 0.7)
    if n > 4:
        w[n // 2] = 0.0
    ends = (w.cumsum(0) / w.sum() * total).round().long().tolist()
    ends[-1] = total
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def _lengths(c):
    """[(queries, keys)] of the sequences: the same for every seed."""
    n, q, k = c["seqs"], c["q"], c["k"]
    if c["layout"] == "dense":
        return [(q, k)] * n
    if c["layout"] == "ragged":
        lq = _parts(q, n, 7)
        return list(zip(lq, lq if k == q else _parts(k, n, 8)))
    full = [max(1, k - (k * 5 * i) // (7 * max(1, n - 1))) for i in range(n)] if n > 1 else [k]
    return [(q, v) for v in full] if c["layout"] == "cache" else [(v, v) for v in full]


# ---------------------------------------------------------------- inputs

def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _rand(g, shape, std, dtype, mean=0.0):
    t = torch.randn(shape, generator=g, device=_dev(), dtype=torch.float32)
    return t.mul_(std).add_(mean).to(dtype)


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=_dev())


def _prepare_attention(c, g):
    D, n, hq, hk, d = DTYPES[c["dtype"]], c["seqs"], c["heads"], c["key_heads"], c["d"]
    lens = _lengths(c)
    lead = lambda m: (m,) if c["layout"] == "ragged" else (n, m)  # noqa: E731
    s = {"lens": lens, "scale": 1.0 / math.sqrt(d)}
    if c["layout"] != "cache" and c["q"] == c["k"]:
        # q, k and v are parts of one projection's output
        qkv = _rand(g, (*lead(c["q"]), (hq + 2 * hk) * d), 1.0, D, 0.02)
        q, k, v = qkv.split([hq * d, hk * d, hk * d], dim=-1)
    else:
        q = _rand(g, (*lead(c["q"]), hq * d), 1.0, D, 0.02)
        k, v = (_rand(g, (*lead(c["k"]), hk * d), 1.0, D, 0.02) for _ in range(2))
    s["q"], s["k"], s["v"] = (t.view(*t.shape[:-1], -1, d) for t in (q, k, v))
    s["opts"] = dict(causal=c["causal"], scale=s["scale"], dropout=c["dropout"],
                     seed=int(torch.randint(0, 2 ** 62, (), generator=g, device=_dev())))
    if c["layout"] == "ragged":
        s["opts"]["q_offsets"] = _starts([a for a, _ in lens])
        s["opts"]["k_offsets"] = _starts([b for _, b in lens])
    elif c["layout"] != "dense":
        s["opts"]["k_lengths"] = torch.tensor([b for _, b in lens], dtype=torch.int32, device=_dev())
        if c["layout"] == "padded":
            s["opts"]["q_lengths"] = s["opts"]["k_lengths"].clone()
    if c["train"]:
        s["dout"] = _rand(g, s["q"].shape, 1.0, D)
    return s


def _prepare_dropout(c, g):
    S, Bt = DTYPES[c["stream"]], DTYPES[c["branch"]]
    shape = (c["rows"], c["d"])
    s = {"x": _rand(g, shape, 0.7, Bt, 0.05), "residual": _rand(g, shape, 2.0, S) if c["residual"] else None,
         "seed": int(torch.randint(0, 2 ** 62, (), generator=g, device=_dev()))}
    if c["train"]:
        s["dy"] = _rand(g, shape, 1.0, S if c["residual"] else Bt)
    return s


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(seed)
    s = (_prepare_attention if case["op"] == "attention" else _prepare_dropout)(case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------- plain forms

def _signed(v):
    return v - (1 << 64) if v >= 1 << 63 else v


def _plain_draws(seed, t):
    """SplitMix64 draw number t (int64 tensor, wrapping arithmetic) of the seed."""
    z = (t + 1) * _signed(0x9E3779B97F4A7C15) + seed
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _signed(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _signed(0x94D049BB133111EB)
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _plain_factor(z, p, width):
    """M of 4 elements for each draw of z [..., n], cut to [..., width]."""
    T = int(p * 65536 + 0.5)
    lanes = torch.arange(0, 64, 16, device=z.device)
    keep = ((z[..., None] >> lanes) & 0xFFFF) >= T
    return keep.flatten(-2)[..., :width] * (65536.0 / (65536 - T))


def _plain_heads(q, k, v, dout, c, factor, scale):
    """One sequence, some key heads: q [Hk][G * nq][d], k and v [Hk][nk][d], factor as P or None."""
    nk = k.shape[1]
    P = torch.matmul(q, k.transpose(1, 2)).mul_(scale)
    nq = P.shape[1] // c["group"]
    if c["causal"]:
        i = torch.arange(nq, device=P.device).repeat(c["group"])[:, None]
        P.masked_fill_(torch.arange(nk, device=P.device)[None, :] > i + (nk - nq), -math.inf)
    top = P.amax(-1, keepdim=True)
    P = P.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    P = P.div_(P.sum(-1, keepdim=True).clamp_min(1e-30))
    Pd = P if factor is None else P * factor
    out = torch.matmul(Pd, v)
    if dout is None:
        return (out,)
    dv = torch.matmul(Pd.transpose(1, 2), dout)
    dP = torch.matmul(dout, v.transpose(1, 2))
    if factor is not None:
        dP.mul_(factor)
    dS = dP.sub_((dP * P).sum(-1, keepdim=True)).mul_(P)
    return out, torch.matmul(dS, k).mul_(scale), torch.matmul(dS.transpose(1, 2), q).mul_(scale), dv


def _plain_attention(s):
    c = dict(s["case"], group=s["case"]["heads"] // s["case"]["key_heads"])
    G, hq, hk, d, o = c["group"], c["heads"], c["key_heads"], c["d"], s["opts"]
    ragged = c["layout"] == "ragged"
    res = {"out": torch.zeros_like(s["q"], memory_format=torch.contiguous_format)}
    if c["train"]:
        for t in "qkv":
            res["d" + t] = torch.zeros_like(s[t], memory_format=torch.contiguous_format)
    aq = ak = 0
    for n, (nq, nk) in enumerate(s["lens"]):
        sq, sk = ((slice(aq, aq + nq), slice(ak, ak + nk)) if ragged else
                  ((n, slice(0, nq)), (n, slice(0, nk))))
        rows = aq if ragged else n * c["q"]
        aq, ak = aq + nq, ak + nk
        if nq == 0 or nk == 0:
            continue
        step = max(1, int(1.5e9 / (nq * nk * G)))
        for h in range(0, hk, step):
            e = min(hk, h + step)
            kh = slice(h, e)
            qs = slice(h * G, e * G)
            heads = lambda t: t.transpose(0, 1).float().reshape(e - h, -1, d)  # noqa: E731
            factor = None
            if c["dropout"]:
                head = torch.arange(h * G, e * G, device=_dev())
                r = (rows + torch.arange(nq, device=_dev()))[None, :] * hq + head[:, None]
                z = _plain_draws(o["seed"], (r.reshape(e - h, -1, 1) << 30)
                                 + torch.arange((nk + 3) // 4, device=_dev()))
                factor = _plain_factor(z, c["dropout"], nk)
            got = _plain_heads(heads(s["q"][sq][:, qs]), heads(s["k"][sk][:, kh]),
                               heads(s["v"][sk][:, kh]),
                               heads(s["dout"][sq][:, qs]) if c["train"] else None, c, factor,
                               s["scale"])
            for name, val, at, which in zip(("out", "dq", "dk", "dv"), got, (sq, sq, sk, sk),
                                            (qs, qs, kh, kh)):
                t = res[name][at]
                t[:, which] = val.view(which.stop - which.start, -1, d).transpose(0, 1).to(t.dtype)
    return res


def _plain_dropout(s):
    c = s["case"]
    n = c["rows"] * c["d"]
    M = _plain_factor(_plain_draws(s["seed"], torch.arange((n + 3) // 4, device=_dev()))[None], c["p"],
                      1 << 62).flatten()[:n].view(c["rows"], c["d"])
    y = s["x"].float() * M
    if s["residual"] is None:
        out = {"y": y.to(s["x"].dtype)}
    else:
        out = {"y": (s["residual"].float() + y).to(s["residual"].dtype)}
    if c["train"]:
        out["dx"] = (s["dy"].float() * M).to(s["x"].dtype)
    return out


# ---------------------------------------------------------------- the package's operators

def _own_attention(s):
    import coo_spmm_sparse_gb300 as sn
    q, k, v = s["q"], s["k"], s["v"]
    out, lse = sn.snack_attention_forward(q, k, v, **s["opts"])
    if not s["case"]["train"]:
        return {"out": out}
    dq, dk, dv = sn.snack_attention_backward(s["dout"], q, k, v, out, lse, **s["opts"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def _own_dropout(s):
    import coo_spmm_sparse_gb300 as sn
    c = s["case"]
    out = {"y": sn.snack_dropout_forward(s["x"], c["p"], s["seed"], residual=s["residual"])}
    if c["train"]:
        out["dx"] = sn.snack_dropout_backward(s["dy"], c["p"], s["seed"], dtype=s["x"].dtype)
    return out


def run(state):
    if state["case"]["op"] == "attention":
        return _own_attention(state) if own else _plain_attention(state)
    return _own_dropout(state) if own else _plain_dropout(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _pairs(nq, nk, causal):
    """Query-key pairs that are seen."""
    if not causal:
        return nq * nk
    first = nk - nq + 1  # keys that query 0 sees
    if first >= 0:
        return nq * first + nq * (nq - 1) // 2
    return nk * (nk + 1) // 2


def work(case):
    c = case
    if c["op"] == "dropout":
        S, Bt, n = SIZE[c["stream"]], SIZE[c["branch"]], c["rows"] * c["d"]
        y = S if c["residual"] else Bt
        nbytes = n * (Bt + y + (S if c["residual"] else 0))
        return {"bytes": nbytes + (n * (y + Bt) if c["train"] else 0), "flops": n * (3 if c["train"] else 2)}
    e, lens, d = SIZE[c["dtype"]], _lengths(c), c["d"]
    q = sum(a for a, _ in lens) * c["heads"] * d * e
    k = sum(b for _, b in lens) * c["key_heads"] * d * e
    pairs = sum(_pairs(a, b, c["causal"]) for a, b in lens) * c["heads"] * d
    nbytes, flops = 2 * q + 2 * k, 4 * pairs
    if c["train"]:  # q, k, v, out and its gradient in again; dq, dk, dv out
        nbytes, flops = nbytes + 4 * q + 4 * k, flops + 10 * pairs
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_factor(seed, first_draw, draws, p):
    """M for 4 * draws elements of each row, from unsigned 64-bit integers on the host."""
    T = round(p * 65536)
    with np.errstate(over="ignore"):
        t = np.asarray(first_draw, dtype=np.uint64)[:, None] + np.arange(draws, dtype=np.uint64)[None, :]
        z = np.uint64(seed) + (t + np.uint64(1)) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    u = np.ascontiguousarray(z).astype("<u8").view("<u2")
    return torch.from_numpy((u >= T).astype(np.float64) / (1.0 - T / 65536.0)).to(_dev())


def _exact_attention(s):
    c, f = s["case"], torch.float64
    G = c["heads"] // c["key_heads"]
    cost = sum(a * b for a, b in s["lens"]) * c["heads"]
    if cost * c["d"] * (12 if c["train"] else 4) > 8e12 or (c["dropout"] and cost > 2e8):
        return None
    dims = ["q", "k", "v"]
    leaf = {t: s[t].to(f) for t in dims}
    res = {"out": torch.zeros(s["q"].shape, dtype=f, device=_dev())}
    if c["train"]:
        res.update({"d" + t: torch.zeros(s[t].shape, dtype=f, device=_dev()) for t in dims})
    start_q = start_k = 0
    for n, (nq, nk) in enumerate(s["lens"]):
        if c["layout"] == "ragged":
            pick = {"q": lambda t, a=start_q, b=nq: t[a: a + b], "k": lambda t, a=start_k, b=nk: t[a: a + b]}
            token = start_q
        else:
            pick = {"q": lambda t, i=n, b=nq: t[i, :b], "k": lambda t, i=n, b=nk: t[i, :b]}
            token = n * c["q"]
        pick["v"] = pick["k"]
        start_q, start_k = start_q + nq, start_k + nk
        seen = torch.ones(nq, nk, dtype=torch.bool, device=_dev())
        if c["causal"]:
            seen = seen.tril(nk - nq)
        some = seen.any(1)
        first = int((~some).sum())  # the rows that see no key come first
        if first == nq:
            continue
        for h in range(c["heads"]):
            qh, kh, vh = (pick[t](leaf[t])[:, h if t == "q" else h // G].clone().requires_grad_(c["train"])
                          for t in dims)
            score = (qh @ kh.T * s["scale"])[first:]
            weights = torch.softmax(torch.where(seen[first:], score, torch.full_like(score, -math.inf)), 1)
            if c["dropout"]:
                rows = [((token + i) * c["heads"] + h) << 30 for i in range(first, nq)]
                weights = weights * _exact_factor(s["opts"]["seed"], rows, (nk + 3) // 4,
                                                  c["dropout"])[:, :nk]
            y = weights @ vh
            pick["q"](res["out"])[first:, h] = y.detach()
            if c["train"]:
                grads = torch.autograd.grad(y, (qh, kh, vh), pick["q"](s["dout"])[first:, h].to(f))
                for t, gr in zip(dims, grads):
                    pick[t](res["d" + t])[:, h if t == "q" else h // G] += gr
    return res


def _exact_dropout(s):
    c, f = s["case"], torch.float64
    n = c["rows"] * c["d"]
    M = _exact_factor(s["seed"], [0], (n + 3) // 4, c["p"])[0, :n].view(c["rows"], c["d"])
    y = s["x"].to(f) * M
    res = {"y": y if s["residual"] is None else s["residual"].to(f) + y}
    if c["train"]:
        res["dx"] = s["dy"].to(f) * M
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_attention if case["op"] == "attention" else _exact_dropout)(s)
