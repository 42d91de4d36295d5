"""Plain 64-bit forms of the block operators, token by token and row by row,
for the tests (torch on the CPU)."""
from __future__ import annotations

import torch


def linattn(q, k, v, log_decay, lens, scale, init=None, do=None, dfinal=None):
    """q, k [T, G, K], v and do [T, H, V] in float64, log_decay [H], lens of the
    packed sequences (from token 0), states [n, H, K, V].  Returns a dict of o
    and final, and with do also dq, dk, dv and dinit."""
    T, H, V = v.shape
    G, K = q.shape[1:]
    n = len(lens)
    lam = torch.exp(log_decay.double())[:, None, None]
    q, k = (x.repeat_interleave(H // G, dim=1) for x in (q, k))
    S0 = torch.zeros(n, H, K, V, dtype=torch.float64) if init is None else init.double()
    o = torch.zeros_like(v)
    final = S0.clone()
    out = {"o": o, "final": final}
    if do is not None:
        R0 = torch.zeros_like(S0) if dfinal is None else dfinal.double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dinit = R0.clone()
    t0 = 0
    for i, L in enumerate(lens):
        S = S0[i]
        for t in range(t0, t0 + L):
            S = lam * S + k[t, :, :, None] * v[t, :, None, :]
            o[t] = scale * torch.einsum("hk,hkv->hv", q[t], S)
            if do is not None:
                dq[t] = scale * torch.einsum("hv,hkv->hk", do[t], S)
        final[i] = S
        if do is not None:
            R = R0[i]
            for t in range(t0 + L - 1, t0 - 1, -1):
                R = R + scale * q[t, :, :, None] * do[t, :, None, :]
                dk[t] = torch.einsum("hkv,hv->hk", R, v[t])
                dv[t] = torch.einsum("hkv,hk->hv", R, k[t])
                R = lam * R
            dinit[i] = R
        t0 += L
    if do is not None:
        out |= {"dq": dq.view(T, G, H // G, K).sum(2), "dk": dk.view(T, G, H // G, K).sum(2),
                "dv": dv, "dinit": dinit}
    return out


def add_norm(x, residual, res_scale, weight, eps, dy=None, dh=None):
    """(y, h), and with dy also the gradients of x, residual, res_scale, weight."""
    h = x if res_scale is None else x * res_scale
    h = h if residual is None else h + residual
    r = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n = h * r
    w = torch.ones_like(h[0]) if weight is None else weight
    out = {"y": n * w, "h": h}
    if dy is not None:
        e = dy * w
        g = r * (e - n * (e * n).mean(-1, keepdim=True))
        g = g if dh is None else g + dh
        out |= {"dresidual": g, "dx": g if res_scale is None else g * res_scale,
                "dres_scale": (g * x).sum(0), "dweight": (dy * n).sum(0)}
    return out


def gated_norm(x, z, weight, eps, group, gate, first, dy=None):
    """y, and with dy also the gradients of x, z and weight."""
    rows, D = x.shape
    x3 = x.view(rows, D // group, group)
    act, dact = torch.ones_like(x3), torch.zeros_like(x3)
    if z is not None:
        z3 = z.view_as(x3)
        sig = 1.0 / (1.0 + torch.exp(-z3))
        act = z3 * sig if gate == "silu" else sig
        dsig = sig * (1.0 - sig)
        dact = sig + z3 * dsig if gate == "silu" else dsig
    w = torch.ones(1, group, dtype=x.dtype) if weight is None else weight.view(-1, group)
    u = x3 * act if first else x3
    r = 1.0 / torch.sqrt((u * u).mean(-1, keepdim=True) + eps)
    n = u * r
    out = {"y": (n * w if first else n * w * act).reshape(rows, D)}
    if dy is not None:
        d3 = dy.view_as(x3)
        dn = d3 if first else d3 * act
        e = dn * w
        du = r * (e - n * (e * n).mean(-1, keepdim=True))
        dz = du * x3 * dact if first else d3 * n * w * dact
        dw = (dn * n).sum(0)
        out |= {"dx": (du * act if first else du).reshape(rows, D), "dz": dz.reshape(rows, D),
                "dweight": dw.sum(0) if weight is not None and weight.numel() == group
                else dw.reshape(-1)}
    return out
