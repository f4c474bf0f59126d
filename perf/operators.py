"""Cases that time the operators around the sparse layers: the norms, gate and
residual of a block, the low-rank adapters beside a projection, and the
gradient norm over many tensors with clipping.

``run`` computes a case in plain torch (32-bit arithmetic, one rounding at the
end), or, with ``own`` set, through the package's entry points.  ``exact``
evaluates the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _norm(name, rows, seqs, d, kind, post, gate, stream, branch, train):
    return {"name": name, "op": "norm", "rows": rows, "seqs": seqs, "d": d, "kind": kind,
            "post": post, "gate": gate, "stream": stream, "branch": branch, "train": train}


def _adapter(name, tokens, requests, adapters, inp, out, rank, dtype, train):
    return {"name": name, "op": "adapter", "tokens": tokens, "requests": requests,
            "adapters": adapters, "inp": inp, "out": out, "rank": rank, "dtype": dtype,
            "train": train}


def _clip(name, what, count, total, spread, src, dst, norm, packed, kept):
    return {"name": name, "op": "clip", "what": what, "count": count, "total": total,
            "spread": spread, "src": src, "dst": dst, "norm": norm, "packed": packed,
            "kept": kept}


def listed():
    return [
        # One decoded token between two blocks of the GPT-2-small-shaped decoder: latency alone.
        _norm("norm_token", 1, 1, 768, "layer", False, "none", "f32", "f32", False),
        # The decoder's training step on its context of 256 tokens: layer norms, no post norm.
        _norm("norm_context_train", 256, 1, 768, "layer", False, "none", "f32", "f32", True),
        # Sequences conditioned by a gate of their own, at a width no vector divides evenly.
        _norm("norm_odd_train", 4095, 15, 1001, "rms", True, "sequence", "f32", "bf16", True),
        # Pre-training of a wide model: norm before and after the block, a learned gate per channel.
        _norm("norm_wide_train", 16384, 4, 4096, "rms", True, "channel", "bf16", "bf16", True),
        # Decoding: 8 requests with an adapter each beside the decoder's attention projection.
        _adapter("adapter_decode", 8, 8, 8, 768, 2304, 8, "f32", False),
        # Decoding at a full batch of a wide model: the adapters' own bytes are the work.
        _adapter("adapter_decode_wide", 64, 64, 48, 4096, 4096, 16, "bf16", False),
        # Prompts of ragged lengths through the decoder's MLP projection, some without an adapter.
        _adapter("adapter_prompts", 4001, 24, 10, 768, 3072, 32, "f32", False),
        # Fine-tuning of several adapters at once on long sequences.
        _adapter("adapter_train", 8192, 16, 4, 4096, 4096, 16, "f32", True),
        # The gradients of adapters on the 48 projections of the decoder: many tensors, few bytes.
        _clip("clip_adapters", "clip", 96, 2_000_000, 0.5, "f32", "f32", "two", False, True),
        # The norm alone, for a log line, over half-precision gradients of very unlike sizes.
        _clip("norm_ragged", "norm", 700, 30_000_001, 2.5, "bf16", "bf16", "two", True, False),
        # The sparse decoder's own gradients: an embedding of 50257 x 768 and many small tensors.
        _clip("clip_decoder", "clip", 148, 40_600_000, 4.0, "f32", "f32", "two", False, True),
        # Half-precision gradients of a large model, clipped into the optimizer's 32-bit buffer.
        _clip("clip_large", "clip", 290, 400_000_003, 1.0, "bf16", "f32", "two", True, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "adapter", "clip"])
    if op == "norm":
        stream, branch = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                     ("f16", "f16"), ("f32", "f16")])
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        train = rng.random() < 0.6
        seqs = rng.choice([1, 1, 2, 3, 8])
        most = 16384 * 4096 // (2 if stream == "f32" else 1)
        rows = seqs * max(1, _log_int(rng, 1, max(2, min(16384, most // d))) // seqs)
        post = rng.random() < 0.6
        gate = rng.choice(["none", "channel", "token", "sequence", "full"])
        if gate == "full":
            rows = max(seqs, rows // 2 // seqs * seqs)
        c = _norm("", rows, seqs, d, rng.choice(["layer", "rms"]), post, gate, stream, branch,
                  train)
    elif op == "adapter":
        train = rng.random() < 0.5
        dtype = rng.choice(["f32", "f32", "bf16", "f16"])
        rank = rng.choice([1, 4, 5, 8, 12, 16, 16, 24, 32, 33, 64])
        inp, out = (_log_int(rng, 64, 4096) for _ in range(2))
        if rng.random() < 0.7:
            inp, out = max(64, inp // 64 * 64), max(64, out // 64 * 64)
        tokens = _log_int(rng, 1, 8192)
        while tokens > 1 and tokens * rank * (inp + out) > 8192 * 16 * 8192:
            tokens //= 2
        requests = min(tokens, _log_int(rng, 1, 64))
        if rng.random() < 0.3:
            tokens = requests
        c = _adapter("", tokens, requests, rng.randint(1, 2 + requests // 2), inp, out, rank,
                     dtype, train)
    else:
        what = rng.choice(["clip", "clip", "norm"])
        src, dst = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
        c = _clip("", what, _log_int(rng, 1, 1200), _log_int(rng, 10_000, 200_000_000),
                  rng.uniform(0.0, 3.0), src, dst if what == "clip" else src,
                  rng.choice(["two", "two", "max"]), rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _rand(g, shape, std, dtype, mean=0.0):
    t = torch.randn(shape, generator=g, device=_dev(), dtype=torch.float32)
    return t.mul_(std).add_(mean).to(dtype)


def _prepare_norm(c, g):
    S, Bt = DTYPES[c["stream"]], DTYPES[c["branch"]]
    d, n = c["d"], c["seqs"]
    t = c["rows"] // n
    shape = (n, t, d)
    x = torch.randn(shape, generator=g, device=_dev())
    x[..., :: max(1, d // 5)] *= 12.0  # the few large channels of a residual stream
    s = {"x": x.to(S), "y": _rand(g, shape, 0.7, Bt, 0.05)}
    gshape = {"none": None, "channel": (d,), "token": (n, t, 1), "sequence": (n, 1, d),
              "full": shape}[c["gate"]]
    s["gate"] = None if gshape is None else _rand(g, gshape, 0.3, Bt, 0.8)
    layer = c["kind"] == "layer"
    f = torch.float32
    s["next_weight"] = _rand(g, (d,), 0.1, f, 1.0)
    s["next_bias"] = _rand(g, (d,), 0.1, f) if layer else None
    s["post_weight"] = _rand(g, (d,), 0.1, f, 1.0) if c["post"] else None
    s["post_bias"] = _rand(g, (d,), 0.1, f) if c["post"] and layer else None
    if c["train"]:
        s["dr"], s["dh"] = _rand(g, shape, 1.0, S), _rand(g, shape, 1.0, Bt)
    s["a"], s["b"], s["eps"] = 1.0, 0.7, 1e-5
    return s


def _prepare_adapter(c, g):
    D = DTYPES[c["dtype"]]
    T, R, N, r = c["tokens"], c["requests"], c["adapters"], c["rank"]
    s = {"X": _rand(g, (T, c["inp"]), 1.0, D),
         "Y": _rand(g, (T, c["out"]), 1.0, D),
         "A": _rand(g, (N, r, c["inp"]), 1.0 / math.sqrt(c["inp"]), D),
         "B": _rand(g, (N, c["out"], r), 1.0 / math.sqrt(r), D),
         "scale": torch.rand(N, generator=g, device=_dev()) + 0.5}
    cut = torch.randperm(max(1, T - 1), generator=g, device=_dev())[: R - 1].sort().values + 1
    ends = torch.tensor([T], device=_dev())
    s["offsets"] = torch.cat([ends * 0, cut, ends]).to(torch.int32)
    # most requests name an adapter, about one in sixteen none (-1)
    pick = torch.randint(0, N, (R,), generator=g, device=_dev())
    bare = torch.rand(R, generator=g, device=_dev()) < 1 / 16
    s["adapter"] = torch.where(bare, torch.full_like(pick, -1), pick).to(torch.int32)
    if c["train"]:
        s["dY"] = _rand(g, (T, c["out"]), 1.0, D)
        s["dX"] = _rand(g, (T, c["inp"]), 1.0, D)
    return s


def _sizes(c, seed):
    """Element counts of the gradient tensors: log-normal with the case's spread, summing to about its total."""
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(torch.randn(c["count"], generator=g, dtype=torch.float64) * c["spread"])
    return [max(1, int(v)) for v in (w / w.sum() * c["total"]).tolist()]


def _views(sizes, dtype, packed, g):
    """One buffer and its tensors: end to end, or each from a multiple of 64 elements."""
    step = [n if packed else (n + 63) // 64 * 64 for n in sizes]
    flat = torch.empty(sum(step), device=_dev(), dtype=dtype)
    if g is None:
        flat.zero_()
    else:
        flat.normal_(0.0, 0.02, generator=g)
    at, out = 0, []
    for n, k in zip(sizes, step):
        out.append(flat[at: at + n])
        at += k
    return flat, out


def _prepare_clip(c, g, seed):
    sizes = _sizes(c, 17)  # the model's tensors: the same for every seed
    # gradients come from autograd, each its own allocation: from a multiple of 64 elements
    _, grads = _views(sizes, DTYPES[c["src"]], False, g)
    s = {"grads": grads, "out": None, "norm_type": math.inf if c["norm"] == "max" else 2.0}
    # about two thirds of the norm that N(0, 0.02) gradients have: the step is clipped
    s["max_norm"] = 0.0627 if c["norm"] == "max" else 0.0137 * math.sqrt(sum(sizes))
    if c["what"] == "clip":
        s["flat"], s["out"] = _views(sizes, DTYPES[c["dst"]], c["packed"], None)
        s["flat_sizes"] = sizes
    if own and c["kept"]:
        import coo_spmm_sparse_gb300 as sn
        s["grad_list"] = sn.snack_tensor_list(s["grads"])
        if s["out"] is not None:
            s["out_list"] = sn.snack_tensor_list(s["out"])
    return s


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(seed)
    if case["op"] == "norm":
        s = _prepare_norm(case, g)
    elif case["op"] == "adapter":
        s = _prepare_adapter(case, g)
    else:
        s = _prepare_clip(case, g, seed)
    s["case"] = case
    return s


# ---------------------------------------------------------------- plain forms

def _plain_stats(v, layer, eps):
    mean = v.mean(-1, keepdim=True) if layer else torch.zeros_like(v[..., :1])
    rstd = torch.rsqrt((v - mean).square().mean(-1, keepdim=True) + eps)
    return (v - mean) * rstd, rstd


def _plain_affine(hat, w, b):
    out = hat if w is None else hat * w
    return out if b is None else out + b


def _plain_norm_back(t, hat, rstd, layer):
    back = t - hat * (t * hat).mean(-1, keepdim=True)
    return rstd * (back - t.mean(-1, keepdim=True) if layer else back)


def _plain_norm(s):
    c = s["case"]
    layer, S, Bt = c["kind"] == "layer", s["x"].dtype, s["y"].dtype
    x, y = s["x"].float(), s["y"].float()
    gate = None if s["gate"] is None else s["gate"].float()
    u, yhat, yr = y, None, None
    if c["post"]:
        yhat, yr = _plain_stats(y, layer, s["eps"])
        u = _plain_affine(yhat, s["post_weight"], s["post_bias"])
    r = s["a"] * x + s["b"] * (u if gate is None else gate * u)
    rhat, rr = _plain_stats(r, layer, s["eps"])
    h = _plain_affine(rhat, s["next_weight"], s["next_bias"])
    out = {"r": r.to(S), "h": h.to(Bt)}
    if not c["train"]:
        return out
    dr, dh = s["dr"].float(), s["dh"].float()
    D = dr + _plain_norm_back(dh * s["next_weight"], rhat, rr, layer)
    out["dx"] = (s["a"] * D).to(S)
    dz = s["b"] * (D if gate is None else gate * D)
    out["dnext_weight"] = (dh * rhat).sum((0, 1))
    if layer:
        out["dnext_bias"] = dh.sum((0, 1))
    if gate is not None:
        full = s["b"] * u * D
        over = {"channel": (0, 1), "token": (2,), "sequence": (1,), "full": ()}[c["gate"]]
        keep = c["gate"] != "channel"
        out["dgate"] = (full.sum(over, keepdim=keep) if over else full).to(Bt)
    if c["post"]:
        out["dy"] = _plain_norm_back(dz * s["post_weight"], yhat, yr, layer).to(Bt)
        out["dpost_weight"] = (dz * yhat).sum((0, 1))
        if layer:
            out["dpost_bias"] = dz.sum((0, 1))
    else:
        out["dy"] = dz.to(Bt)
    return out


def _token_mask(s):
    """[T][N]: scale of adapter n where token t's request names it, else 0; and the same as truth values."""
    T, N = s["X"].shape[0], s["A"].shape[0]
    t = torch.arange(T, device=s["X"].device, dtype=torch.int32)
    request = torch.searchsorted(s["offsets"][1:].contiguous(), t, right=True)
    of = s["adapter"][request].long()
    hit = of[:, None] == torch.arange(N, device=of.device)[None, :]
    return hit * s["scale"], hit


def _plain_adapter(s):
    # every token through every adapter at once, then the rows' own picked out: two large products
    D = s["X"].dtype
    X, Y, A, B = (s[k].float() for k in ("X", "Y", "A", "B"))
    T, (N, r, inp), out = X.shape[0], A.shape, B.shape[1]
    weight, hit = _token_mask(s)
    Aw = A.reshape(N * r, inp)
    Bw = B.permute(1, 0, 2).reshape(out, N * r)
    H = (X @ Aw.T).view(T, N, r)
    sH = (H * weight[:, :, None]).view(T, N * r)
    res = {"Y": s["Y"].copy_(Y + sH @ Bw.T)}
    if not s["case"]["train"]:
        return res
    dY, dX = s["dY"].float(), s["dX"].float()
    dH = ((dY @ Bw).view(T, N, r) * weight[:, :, None]).view(T, N * r)
    res["dX"] = s["dX"].copy_(dX + dH @ Aw)
    res["dA"] = (dH.T @ X).view(N, r, inp).to(D)
    res["dB"] = (dY.T @ sH).view(out, N, r).permute(1, 0, 2).to(D).contiguous()
    return res


def _plain_clip(s):
    c = s["case"]
    flat = torch.cat([g.float() for g in s["grads"]])
    total = flat.abs().max() if c["norm"] == "max" else flat.square().sum().sqrt()
    if c["what"] == "norm":
        return {"norm": total}
    coef = (s["max_norm"] / (total + 1e-6)).clamp(max=1.0)
    torch._foreach_copy_(s["out"], list((flat * coef).split(s["flat_sizes"])))
    return {"norm": total, "flat": s["flat"]}


# ---------------------------------------------------------------- the package's operators

def _own_norm(s):
    import coo_spmm_sparse_gb300 as sn
    c = s["case"]
    opts = dict(kind=c["kind"], post_norm=c["post"], post_weight=s["post_weight"],
                post_bias=s["post_bias"], gate=s["gate"], residual_scale=s["a"],
                branch_scale=s["b"], next_weight=s["next_weight"], next_bias=s["next_bias"],
                eps=s["eps"])
    r, h, stats = sn.snack_residual_norm_forward(s["x"], s["y"], **opts)
    out = {"r": r, "h": h}
    if c["train"]:
        out.update(sn.snack_residual_norm_backward(s["dr"], s["dh"], s["x"], s["y"], stats, **opts))
    return out


def _own_adapter(s):
    import coo_spmm_sparse_gb300 as sn
    args = (s["A"], s["B"], s["offsets"], s["adapter"], s["scale"])
    Y, H = sn.snack_adapter_forward(s["X"], *args, s["Y"])
    out = {"Y": Y}
    if s["case"]["train"]:
        out["dX"], out["dA"], out["dB"] = sn.snack_adapter_backward(s["X"], s["dY"], *args, H,
                                                                   dX=s["dX"])
    return out


def _own_clip(s):
    import coo_spmm_sparse_gb300 as sn
    grads = s.get("grad_list", s["grads"])
    if s["case"]["what"] == "norm":
        return {"norm": sn.snack_grad_norm(grads, s["norm_type"])}
    total = sn.snack_clip_grad_norm(grads, s["max_norm"], s["norm_type"],
                                    out=s.get("out_list", s["out"]))
    return {"norm": total, "flat": s["flat"]}


def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    if op == "adapter":
        return _own_adapter(state) if own else _plain_adapter(state)
    return _own_clip(state) if own else _plain_clip(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "norm":
        S, Bt, n, d = SIZE[c["stream"]], SIZE[c["branch"]], c["rows"] * c["d"], c["d"]
        gate = Bt * {"none": 0, "channel": d, "token": c["rows"], "sequence": c["seqs"] * d,
                     "full": n}[c["gate"]]
        params = 4 * d * ((2 if c["kind"] == "layer" else 1) * (2 if c["post"] else 1))
        nbytes, flops = n * (2 * S + 2 * Bt) + gate + params, n * (18 if c["post"] else 12)
        if c["train"]:  # x, y, the gate and the weights again, dr and dh in; dx, dy, dgate, dweights out
            nbytes += n * (3 * S + 3 * Bt) + 2 * gate + 2 * params
            flops += n * (36 if c["post"] else 20)
        return {"bytes": nbytes, "flops": flops}
    if c["op"] == "adapter":
        e = SIZE[c["dtype"]]
        T, inp, out, r = c["tokens"], c["inp"], c["out"], c["rank"]
        used = min(c["adapters"], c["requests"]) * r * (inp + out) * e
        nbytes, flops = T * (inp + 2 * out) * e + used, 2 * T * r * (inp + out)
        if c["train"]:  # X, dY and dX in, dX out; the adapters in, their gradients out
            nbytes += T * (3 * inp + out) * e + used + c["adapters"] * r * (inp + out) * e
            flops += 4 * T * r * (inp + out)
        return {"bytes": nbytes, "flops": flops}
    n = sum(_sizes(c, 17))
    return {"bytes": n * (SIZE[c["src"]] + (SIZE[c["dst"]] if c["what"] == "clip" else 0)),
            "flops": n * (3 if c["what"] == "clip" else 2)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(s):
    c, f = s["case"], torch.float64
    leaf = {k: s[k].to(f).requires_grad_(c["train"]) for k in
            ("x", "y", "gate", "post_weight", "post_bias", "next_weight", "next_bias")
            if s[k] is not None}

    def norm(v, which):
        if c["kind"] == "layer":
            v = v - v.mean(-1, keepdim=True)
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + s["eps"])
        if which + "_weight" in leaf:
            v = v * leaf[which + "_weight"]
        return v + leaf[which + "_bias"] if which + "_bias" in leaf else v

    u = norm(leaf["y"], "post") if c["post"] else leaf["y"]
    if "gate" in leaf:
        u = leaf["gate"] * u
    r = s["a"] * leaf["x"] + s["b"] * u
    h = norm(r, "next")
    res = {"r": r.detach(), "h": h.detach()}
    if c["train"]:
        grads = torch.autograd.grad([r, h], list(leaf.values()), [s["dr"].to(f), s["dh"].to(f)])
        res.update({"d" + k: v for k, v in zip(leaf, grads)})
    return res


def _exact_adapter(s):
    f = torch.float64
    X, Y, A, B = (s[k].to(f) for k in ("X", "Y", "A", "B"))
    train = s["case"]["train"]
    if train:
        dY, dX = s["dY"].to(f), s["dX"].to(f)
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    off, which, scale = s["offsets"].tolist(), s["adapter"].tolist(), s["scale"].double().tolist()
    for i, n in enumerate(which):
        t = slice(off[i], off[i + 1])
        if n < 0:
            continue
        H = torch.einsum("ti,ri->tr", X[t], A[n])
        Y[t] += scale[n] * torch.einsum("tr,or->to", H, B[n])
        if train:
            dH = scale[n] * torch.einsum("to,or->tr", dY[t], B[n])
            dX[t] += torch.einsum("tr,ri->ti", dH, A[n])
            dA[n] += torch.einsum("tr,ti->ri", dH, X[t])
            dB[n] += scale[n] * torch.einsum("to,tr->or", dY[t], H)
    return {"Y": Y, "dX": dX, "dA": dA, "dB": dB} if train else {"Y": Y}


def _exact_clip(s):
    f = torch.float64
    if s["case"]["norm"] == "max":
        total = torch.stack([g.to(f).abs().max() for g in s["grads"]]).max()
    else:
        total = torch.stack([g.to(f).square().sum() for g in s["grads"]]).sum().sqrt()
    if s["out"] is None:
        return {"norm": total}
    coef = min(1.0, s["max_norm"] / (float(total) + 1e-6))
    base, flat = s["flat"].data_ptr(), torch.zeros(s["flat"].numel(), dtype=f, device=_dev())
    for g, o in zip(s["grads"], s["out"]):
        at = (o.data_ptr() - base) // o.element_size()
        flat[at: at + g.numel()] = g.to(f) * coef
    return {"norm": total, "flat": flat}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "adapter": _exact_adapter, "clip": _exact_clip}[case["op"]](s)
