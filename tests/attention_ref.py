"""64-bit reference of the attention, and the bounds its outputs are held to.

With A[i, j] = |scale| * sum |q k|, a score is off by at most
d_i = 2^-18 * max_j A[i, j]: products of 128 terms split in two tf32 parts
(2^-22 left out) or exact (16-bit types), summed in 32 bits by steps that cut
off (up to 48 steps of 2^-23), and the exponent's own rounding.  A
probability is then off by a share 2 * d_i (numerator and sum) and 2^-16 (the
sum, the exponential), and, in 16-bit types, by u(T) for the rounding before
the second product (float16: at least 2^-25 of the row's largest).  Sums over
keys or queries of any magnitude add 1e-5 of their terms.  delta is a sum
over the rounded out.  The last rounding adds u(T) of the value."""

import torch

F64 = torch.float64
U = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-30, torch.bfloat16: 1e-30, torch.float16: 2.0 ** -25}
GOLDEN, M1, M2 = 0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB


def draw(seed, t):
    """SplitMix64 draw number t, in Python's integers."""
    mask = (1 << 64) - 1
    z = (seed + (t + 1) * GOLDEN) & mask
    z = ((z ^ (z >> 30)) * M1) & mask
    z = ((z ^ (z >> 27)) * M2) & mask
    return z ^ (z >> 31)


def draws(seed, t):
    """The same for an int64 tensor of numbers (wrapping arithmetic)."""
    s = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
    r = lambda z, n: (z >> n) & ((1 << (64 - n)) - 1)  # noqa: E731
    z = (t + 1) * s(GOLDEN) + s(seed % (1 << 64))
    z = (z ^ r(z, 30)) * s(M1)
    z = (z ^ r(z, 27)) * s(M2)
    return z ^ r(z, 31)


def mask_of(seed, first, n, p):
    """M (float64) of n elements for each row of `first`, the number of its first draw."""
    T = round(p * 65536)
    c = torch.arange((n + 3) // 4, device=first.device)
    z = draws(seed, first[..., None] + c)
    u = (z[..., None] >> torch.arange(0, 64, 16, device=first.device)) & 0xFFFF
    return (u >= T).to(F64).flatten(-2)[..., :n] * (65536.0 / (65536 - T))


def one_sequence(q, k, v, *, causal, scale, M=None, dout=None, dtype=None):
    """q [H, nq, d], k and v [H, nk, d] (heads repeated): name -> (value, bound)."""
    u, tiny = U[dtype], TINY[dtype]
    half = dtype == torch.float16
    q, k, v = (t.to(F64) for t in (q, k, v))
    nq, nk = q.shape[1], k.shape[1]
    s = scale * q @ k.mT
    A = abs(scale) * q.abs() @ k.abs().mT
    seen = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
    if causal:
        seen = seen.tril(nk - nq)
    s = torch.where(seen, s, torch.full_like(s, -torch.inf))
    lse = torch.logsumexp(s, -1) if nk else torch.full_like(s.sum(-1), -torch.inf)
    P = torch.where(lse[..., None] == -torch.inf, torch.zeros_like(s), torch.exp(s - lse[..., None]))
    d = (2.0 ** -18 * torch.where(seen, A, torch.zeros_like(A))).amax(-1, keepdim=True) if nk \
        else torch.zeros_like(lse)[..., None]
    share = 2 * d + 2.0 ** -16 + 1e-5
    M = torch.ones_like(P) if M is None else M
    PM = P * M
    low = 2.0 ** -25 * (M * seen * P.amax(-1, keepdim=True)) if half and nk else torch.zeros_like(P)
    out = PM @ v
    e_out = (PM * (share + u) + low) @ v.abs() + u * out.abs() + tiny
    res = {"out": (out, e_out), "lse": (lse, d[..., 0] + 2.0 ** -16 + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0))}
    if dout is None:
        return res
    dout = dout.to(F64)
    dP = dout @ v.mT
    delta = (dout * out).sum(-1, keepdim=True)
    dS = P * (M * dP - delta)
    e_dP = 2.0 ** -18 * M * (dout.abs() @ v.abs().mT)
    e_delta = ((dout.abs() * e_out).sum(-1, keepdim=True) + 1e-5 * (dout.abs() * out.abs()).sum(-1, keepdim=True))
    e_dS = dS.abs() * (share + u) + P * (e_dP + e_delta)
    # Operands of the backward products may be float16 (32-bit floats in two parts): dS is scaled
    # so that its bound 2 d max|dout| max|v| max(M) is at least 2^13, and half a step of the
    # smallest float16 is 2^-25: 2^-38 of the bound.  P is taken 2^14 fold: 2^-39.
    top = dout.abs().max() * v.abs().max() * M.max() if dout.numel() and v.numel() else 0.0
    e_dS = e_dS + seen * (2 * q.shape[-1] * top * 2.0 ** -38)
    low = 2.0 ** -39 * seen
    res["dq"] = (scale * dS @ k, abs(scale) * (e_dS + 1e-5 * dS.abs()) @ k.abs())
    res["dk"] = (scale * dS.mT @ q, abs(scale) * (e_dS + 1e-5 * dS.abs()).mT @ q.abs())
    res["dv"] = (PM.mT @ dout, (PM * (share + u) + low * M).mT @ dout.abs())
    for n in ("dq", "dk", "dv"):
        val, e = res[n]
        res[n] = (val, e + tiny)
    return res


def attention(q, k, v, *, causal=True, scale=None, q_offsets=None, k_offsets=None, q_lengths=None,
              k_lengths=None, dropout=0.0, seed=0, dout=None):
    """name -> (value, bound), laid out as the operator's results (rounding to the type included)."""
    H, Hk, d, dtype, dev = q.shape[-2], k.shape[-2], q.shape[-1], q.dtype, q.device
    G = H // Hk
    scale = d ** -0.5 if scale is None else scale
    res = {n: [torch.zeros(t.shape, dtype=F64, device=dev) for _ in range(2)]
           for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", k))}
    rows = q.shape[:-2].numel()
    lse = [torch.full((H, rows), -torch.inf, dtype=F64, device=dev), torch.zeros(H, rows, dtype=F64, device=dev)]
    n = q_offsets.numel() - 1 if q_offsets is not None else q.shape[0]

    def part(t, off, length, i):
        if off is not None:
            return slice(int(off[i]), int(off[i + 1])), int(off[i])
        size = t.shape[1] if length is None else int(length[i])
        return (i, slice(0, size)), i * t.shape[1]

    for i in range(n):
        a, row = part(q, q_offsets, q_lengths, i)
        b, _ = part(k, k_offsets, k_lengths, i)
        qs, ks, vs = q[a].transpose(0, 1), k[b].transpose(0, 1), v[b].transpose(0, 1)
        nq, nk = qs.shape[1], ks.shape[1]
        M = None
        if dropout:
            number = (row + torch.arange(nq, device=dev)) * H + torch.arange(H, device=dev)[:, None]
            M = mask_of(seed, number << 30, nk, dropout)
        got = one_sequence(qs, ks.repeat_interleave(G, 0), vs.repeat_interleave(G, 0), causal=causal,
                           scale=scale, M=M, dout=None if dout is None else dout[a].transpose(0, 1), dtype=dtype)
        for name, (val, e) in got.items():
            for j, t in enumerate((val, e)):
                if name == "lse":
                    lse[j][:, row: row + nq] = t
                elif name in ("dk", "dv"):
                    res[name][j][b] = t.view(Hk, G, nk, d).sum(1).transpose(0, 1)
                else:
                    res[name][j][a] = t.transpose(0, 1)
    for name in ("dq", "dk", "dv"):
        res[name][1] += U[dtype] * res[name][0].abs()
    if dout is None:
        res = {"out": res["out"]}
    res["lse"] = [t.view(H, *q.shape[:-2]) for t in lse]
    return res


def assert_within(got, want):
    for name, g in got.items():
        ref, bound = want[name]
        g = g.detach().to(F64)
        assert g.shape == ref.shape, (name, g.shape, ref.shape)
        bad = ~(((g - ref).abs() <= bound * 1.01) | (g == ref))
        assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist(),
                               float((g - ref).abs().nan_to_num(1e30).max()), float(bound.max()))
