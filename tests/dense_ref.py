"""64-bit references of the dense operators, and the bounds their outputs are held to.

Every reference returns, beside a value, S: the sum of the magnitudes of the
terms that make it up.  An output of type T may be off by
1e-5 * S + u(T) * |value| + tiny(T): 1e-5 of the terms is the rule of the
sparse products' tests (168 roundings of 2^-24, for sums that run through a
warp, a block and a few partials), u(T) the half unit of the one rounding to
T (2^-8 for bfloat16, 2^-11 for float16; float32's is in the 1e-5), tiny(T)
half of the smallest float16 subnormal."""

import torch

F64 = torch.float64
U = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def assert_within(name, got, want, S, slack=1e-5):
    ref = want.to(F64).cpu()
    g = got.detach().to(F64).cpu()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    bound = slack * S.to(F64).cpu() + U[got.dtype] * 1.01 * ref.abs() + TINY[got.dtype]
    err = (g - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float((err - bound).max()), float(err.max()))


def _stats(v, layer, eps):
    mean = v.mean(-1, keepdim=True) if layer else torch.zeros_like(v[..., :1])
    rstd = 1.0 / torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + eps)
    return mean, rstd


def _one(t, like):
    return torch.ones_like(like) if t is None else t


def _zero(t, like):
    return torch.zeros_like(like) if t is None else t


def residual_norm(x, y, *, kind, post_norm=False, post_weight=None, post_bias=None, gate=None,
                  residual_scale=1.0, branch_scale=1.0, next_norm=True, next_weight=None,
                  next_bias=None, eps=1e-5, dr=None, dh=None):
    """dict name -> (value, S) of the outputs and, with dr / dh, of the gradients."""
    c = lambda t: None if t is None else t.detach().to(F64).cpu()  # noqa: E731
    x, y, gate, dr, dh = c(x), c(y), c(gate), c(dr), c(dh)
    pw, pb, nw, nb = c(post_weight), c(post_bias), c(next_weight), c(next_bias)
    layer = kind == "layer"
    a, b = residual_scale, branch_scale
    one = torch.ones_like(x)
    res = {}
    g = one if gate is None else gate.expand_as(x)
    r, Sr = a * x, (a * x).abs()
    if y is not None:
        if post_norm:
            ym, yr = _stats(y, layer, eps)
            yhat, Syhat = (y - ym) * yr, (y.abs() + ym.abs()) * yr
            u = yhat * _one(pw, x) + _zero(pb, x)
            Su = Syhat * _one(pw, x).abs() + _zero(pb, x).abs()
        else:
            u, Su = y, y.abs()
        r, Sr = r + b * g * u, Sr + (b * g).abs() * Su
    res["r"] = (r, Sr)
    if next_norm:
        m, rs = _stats(r, layer, eps)
        rhat, Srhat = (r - m) * rs, (Sr + m.abs()) * rs
        res["h"] = (rhat * _one(nw, x) + _zero(nb, x),
                    Srhat * _one(nw, x).abs() + _zero(nb, x).abs())
    if dr is None and dh is None:
        return res
    D, SD = (torch.zeros_like(x),) * 2
    if dr is not None:
        D, SD = dr, dr.abs()

    def back(t, St, hat, Shat, rstd):
        v = t - hat * (t * hat).mean(-1, keepdim=True)
        S = St + Shat * (St * Shat).mean(-1, keepdim=True)
        if layer:
            v, S = v - t.mean(-1, keepdim=True), S + St.mean(-1, keepdim=True)
        return rstd * v, rstd * S

    over = tuple(range(x.dim() - 1))
    if dh is not None:
        t = dh * _one(nw, x)
        v, S = back(t, t.abs(), rhat, Srhat, rs)
        D, SD = D + v, SD + S
        if nw is not None:
            res["dnext_weight"] = ((dh * rhat).sum(over), (dh.abs() * Srhat).sum(over))
        if nb is not None:
            res["dnext_bias"] = (dh.sum(over), dh.abs().sum(over))
    else:
        for k, t in (("dnext_weight", nw), ("dnext_bias", nb)):
            if t is not None:
                res[k] = (torch.zeros_like(t), torch.zeros_like(t))
    res["dx"] = (a * D, abs(a) * SD)
    if y is None:
        return res
    dz, Sdz = b * g * D, (b * g).abs() * SD
    if post_norm:
        p, Sp = dz * _one(pw, x), Sdz * _one(pw, x).abs()
        res["dy"] = back(p, Sp, yhat, Syhat, yr)
        if pw is not None:
            res["dpost_weight"] = ((dz * yhat).sum(over), (Sdz * Syhat).sum(over))
        if pb is not None:
            res["dpost_bias"] = (dz.sum(over), Sdz.sum(over))
    else:
        res["dy"] = (dz, Sdz)
    if gate is not None:
        full, S = b * u * D, abs(b) * Su * SD
        if gate.shape != x.shape:
            dims = [i - gate.dim() + x.dim() for i in range(gate.dim()) if gate.shape[i] == 1
                    and x.shape[i - gate.dim() + x.dim()] != 1]
            dims += list(range(x.dim() - gate.dim()))
            if dims:
                full, S = full.sum(dims, keepdim=True), S.sum(dims, keepdim=True)
            full, S = full.reshape(gate.shape), S.reshape(gate.shape)
        res["dgate"] = (full, S)
    return res


def adapter(X, Y, A, B, offsets, which, scale, dY=None, dX=None):
    """dict name -> (value, S) for Y, H and, with dY, dX / dA / dB."""
    c = lambda t: t.detach().to(F64).cpu()  # noqa: E731
    X, Y, A, B = c(X), c(Y), c(A), c(B)
    N, r, inp = A.shape
    T = X.shape[0]
    sc = c(scale).tolist() if isinstance(scale, torch.Tensor) else [float(scale)] * N
    H, SH = torch.zeros(T, r, dtype=F64), torch.zeros(T, r, dtype=F64)
    Yo, SY = Y.clone(), Y.abs()
    if dY is not None:
        dY = c(dY)
        dXo = torch.zeros_like(X) if dX is None else c(dX)
        SX = dXo.abs()
        dXo = dXo.clone()
        dA, SA, dB, SB = (torch.zeros_like(t) for t in (A, A, B, B))
    off = offsets.tolist()
    for i, n in enumerate(which.tolist()):
        t0, t1 = off[i], off[i + 1]
        if not 0 <= n < N or t1 <= t0:
            continue
        s = slice(t0, t1)
        H[s], SH[s] = X[s] @ A[n].T, X[s].abs() @ A[n].abs().T
        Yo[s] += sc[n] * (H[s] @ B[n].T)
        SY[s] += abs(sc[n]) * (SH[s] @ B[n].abs().T)
        if dY is not None:
            dH, SdH = sc[n] * (dY[s] @ B[n]), abs(sc[n]) * (dY[s].abs() @ B[n].abs())
            dXo[s] += dH @ A[n]
            SX[s] += SdH @ A[n].abs()
            dA[n] += dH.T @ X[s]
            SA[n] += SdH.T @ X[s].abs()
            dB[n] += sc[n] * (dY[s].T @ H[s])
            SB[n] += abs(sc[n]) * (dY[s].abs().T @ SH[s])
    res = {"Y": (Yo, SY), "H": (H, SH)}
    if dY is not None:
        res.update(dX=(dXo, SX), dA=(dA, SA), dB=(dB, SB))
    return res
