"""Plain 64-bit forms of the operators around a selective state space, token by token,
for the tests (torch on the CPU), and the comparison with them.

With ``size`` every term is taken by its absolute value: what a result's sums add up to
before anything cancels, which is what their roundings are relative to."""
from __future__ import annotations

import torch


def _cuts(lens):
    at = 0
    for i, n in enumerate(lens):
        yield i, at, at + n
        at += n


def conv(x, weight, bias, lens, silu, init=None, dy=None, dfinal=None, size=False):
    """x, dy [T, D], weight [D, W], states [n, W-1, D], all float64."""
    n, W, D = len(lens), weight.shape[1], x.shape[1]
    init0 = torch.zeros(n, W - 1, D, dtype=torch.float64) if init is None else init
    b = torch.zeros(D, dtype=torch.float64) if bias is None else bias
    y, final = torch.zeros_like(x), torch.zeros_like(init0)
    dx, dinit = torch.zeros_like(x), torch.zeros_like(init0)
    dw, db = torch.zeros_like(weight), torch.zeros_like(b)

    def mag(t):
        return t.abs() if size else t

    for i, a, e in _cuts(lens):
        ext = torch.cat([init0[i], x[a:e]])
        pre = b + sum(weight[:, k] * ext[k:k + e - a] for k in range(W))
        sig = torch.sigmoid(pre)
        summed = mag(b) + sum(mag(weight[:, k]) * mag(ext[k:k + e - a]) for k in range(W))
        y[a:e] = summed * (sig if silu else 1.0)
        final[i] = mag(ext[e - a:])
        if dy is not None:
            slope = sig * (1 + pre * (1 - sig)) if silu else torch.ones_like(pre)
            if size and silu:    # the slope's own error: at most 1/2 of the sum's
                slope = slope.abs() + summed
            g = mag(dy[a:e]) * slope
            dext = torch.zeros(W - 1 + e - a, D, dtype=torch.float64)
            for k in range(W):
                dext[k:k + e - a] += mag(weight[:, k]) * g
                dw[:, k] += (g * mag(ext[k:k + e - a])).sum(0)
            db += g.sum(0)
            if dfinal is not None:
                dext[e - a:] += mag(dfinal[i])
            dinit[i], dx[a:e] = dext[:W - 1], dext[W - 1:]
    out = {"y": y, "final": final}
    return out | ({"dx": dx, "dweight": dw, "dbias": db, "dinit": dinit} if dy is not None else {})


def scan(x, dt, A, B, C, D, z, bias, lens, softplus=True, init=None, dy=None, dfinal=None,
         size=False):
    """x, dt, z, dy [T, D], A [D, N], B, C [T, G, N], states [n, D, N], all float64."""
    T, dim = x.shape
    N, G, n = A.shape[1], B.shape[1], len(lens)

    def mag(t):
        return t.abs() if size else t

    raw = dt if bias is None else dt + bias
    delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())) if softplus else raw
    decay = torch.exp(delta[..., None] * A)
    x, B, C, delta = mag(x), mag(B), mag(C), mag(delta)
    wide = dim // G
    Bw, Cw = (t.repeat_interleave(wide, dim=1) for t in (B, C))
    skip = torch.zeros(dim, dtype=torch.float64) if D is None else mag(D)
    if z is None:
        gate, slope = torch.ones_like(x), None
    else:
        sig = torch.sigmoid(z)
        gate = mag(z * sig)
        slope = mag(sig) + mag(z * sig * (1 - sig)) if size else sig * (1 + z * (1 - sig))
    h0 = torch.zeros(n, dim, N, dtype=torch.float64) if init is None else mag(init)
    hs = torch.zeros(T, dim, N, dtype=torch.float64)
    before, final = torch.zeros_like(hs), h0.clone()
    u = torch.zeros_like(x)
    for i, a, e in _cuts(lens):
        h = h0[i]
        for t in range(a, e):
            before[t] = h
            h = decay[t] * h + (delta[t] * x[t])[:, None] * Bw[t]
            hs[t] = h
        final[i] = h
    u = (hs * Cw).sum(-1) + skip * x
    out = {"y": u * gate, "final": final}
    if dy is None:
        return out
    dy = mag(dy)
    du = dy * gate
    R0 = torch.zeros_like(h0) if dfinal is None else mag(dfinal)
    R = torch.zeros_like(hs)
    dinit = R0.clone()
    for i, a, e in _cuts(lens):
        r = R0[i]
        for t in range(e - 1, a - 1, -1):
            r = r + Cw[t] * du[t][:, None]
            R[t] = r
            r = decay[t] * r
        dinit[i] = r
    kept = R * decay * before
    inner = (R * Bw).sum(-1)
    ddt = x * inner + (kept * mag(A)).sum(-1)
    if softplus:
        ddt = ddt * torch.sigmoid(raw)
    out |= {"dx": delta * inner + skip * du, "ddt": ddt, "dA": (kept * delta[..., None]).sum(0),
            "dB": (R * (delta * x)[..., None]).view(T, G, wide, N).sum(2),
            "dC": (hs * du[..., None]).view(T, G, wide, N).sum(2),
            "dD": (du * x).sum(0), "ddt_bias": ddt.sum(0), "dinit": dinit}
    if z is not None:
        out["dz"] = dy * u * slope
    return out


E4M3 = torch.float8_e4m3fn


def quant(x, res, scale, weight, eps, group, dtype):
    """Rows in float64: the stream, the codes' values, the scales, and y."""
    h = x if scale is None else x * scale
    h = h if res is None else h + res
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    y = y if weight is None else y * weight
    yg = y.unflatten(-1, (-1, group))
    top = 448.0 if dtype == E4M3 else 127.0
    most = yg.abs().amax(-1, keepdim=True)
    v = torch.where(most >= 1e-30, yg * (top / most), torch.zeros_like(yg))
    if dtype == E4M3:
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        codes = torch.round(v / unit) * unit
    else:
        codes = torch.round(v)
    return {"h": h, "y": y, "codes": codes.flatten(-2), "v": v.flatten(-2),
            "scales": most[..., 0] / top}


# Which dimensions of a result a norm is taken over: channels (and states) are looked
# at one by one, so that a large one does not hide another's mistakes.
OVER = {"y": 0, "dx": 0, "ddt": 0, "dz": 0, "dB": 0, "dC": 0, "final": -1, "dinit": -1,
        "dA": -1, "dD": None, "ddt_bias": None, "dweight": -1, "dbias": None}


def check(got, ref, size, sums, own=()):
    """The 2-norm of each result's error, per channel, is at most sums times that of the
    same result of absolute values, and 2^-8 of the result for what is rounded to bf16 at
    the end (half a step).  ``own``: results that must be equal."""
    worst = {}
    for n, g in got.items():
        r, a = ref[n], size[n]
        rounded = g.dtype == torch.bfloat16
        g = g.double().cpu()
        assert g.shape == r.shape, (n, g.shape, r.shape)
        assert torch.isfinite(g).all(), n
        if n in own:
            assert torch.equal(g, r), n
            continue
        over = OVER[n]
        err, r, a = ((t.abs() if over is None else t.square().sum(over).sqrt())
                     for t in (g - r, r, a))
        tol = sums * a + (2.0 ** -8 * r if rounded else 0.0) + 1e-30
        worst[n] = float((err / tol).max()) if err.numel() else 0.0
        bad = (err > tol).nonzero()
        assert bad.numel() == 0, (n, bad[0].tolist(), float(err[tuple(bad[0])]),
                                  float(tol[tuple(bad[0])]))
    return worst
