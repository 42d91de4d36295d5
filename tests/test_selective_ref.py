"""The plain forms that the GPU tests compare with (selective_ref.py), themselves compared
with the same recurrences under automatic differentiation and with differences.  No
GPU."""
import pytest
import torch

import selective_ref as ref


def close(a, b):
    assert a.shape == b.shape and float((a - b).abs().max()) <= 1e-11 * (1 + float(b.abs().max()))


def normal(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv(W, silu):
    g = torch.Generator().manual_seed(W)
    lens, D = [5, 0, 1, 2, 9], 3
    T, n = sum(lens), len(lens)
    x, w, b = normal(g, T, D), normal(g, D, W), normal(g, D)
    init, dy, dfinal = normal(g, n, W - 1, D), normal(g, T, D), normal(g, n, W - 1, D)
    leaves = [t.requires_grad_() for t in (x, w, b, init)]
    ys, fs = [], []
    for i, a, e in ref._cuts(lens):
        ext = torch.cat([init[i], x[a:e]])
        pre = torch.stack([b + sum(w[:, k] * ext[t + k] for k in range(W)) for t in range(e - a)]) \
            if e > a else x[a:e] * 0
        ys.append(pre * torch.sigmoid(pre) if silu else pre)
        fs.append(ext[e - a:])
    y, final = torch.cat(ys), torch.stack(fs)
    grads = torch.autograd.grad([y, final], leaves, [dy, dfinal])
    x, w, b, init = (t.detach() for t in leaves)
    out = ref.conv(x, w, b, lens, silu, init, dy, dfinal)
    for n_, t in zip(("y", "final", "dx", "dweight", "dbias", "dinit"), (y, final, *grads)):
        close(out[n_], t.detach())


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_scan(gated, softplus):
    g = torch.Generator().manual_seed(7)
    lens, D, N, G = [4, 0, 1, 6], 6, 3, 2
    T, n = sum(lens), len(lens)
    x, dt = normal(g, T, D), normal(g, T, D)
    if not softplus:
        dt = dt.abs()
    z = normal(g, T, D) if gated else None
    A, B, C = -normal(g, D, N).abs(), normal(g, T, G, N), normal(g, T, G, N)
    skip, bias = normal(g, D), normal(g, D) * (1 if softplus else 0)
    init, dy, dfinal = normal(g, n, D, N), normal(g, T, D), normal(g, n, D, N)
    names = ["x", "dt", "A", "B", "C", "D", "dt_bias", "init"] + (["z"] if gated else [])
    leaves = [t.requires_grad_() for t in (x, dt, A, B, C, skip, bias, init)]
    leaves += [z.requires_grad_()] if gated else []

    def run(x, dt, A, B, C, skip, bias, init, z=None):
        raw = dt + bias
        delta = torch.nn.functional.softplus(raw) if softplus else raw
        ys, fs = [], []
        for i, a, e in ref._cuts(lens):
            h = init[i]
            for t in range(a, e):
                h = torch.exp(delta[t, :, None] * A) * h + (delta[t] * x[t])[:, None] \
                    * B[t].repeat_interleave(D // G, 0)
                u = (h * C[t].repeat_interleave(D // G, 0)).sum(-1) + skip * x[t]
                ys.append(u if z is None else u * torch.nn.functional.silu(z[t]))
            fs.append(h)
        return torch.stack(ys), torch.stack(fs)

    y, final = run(*leaves)
    grads = dict(zip(names, torch.autograd.grad([y, final], leaves, [dy, dfinal])))
    plain = [t.detach() for t in leaves]
    x, dt, A, B, C, skip, bias, init = plain[:8]
    out = ref.scan(x, dt, A, B, C, skip, plain[8] if gated else None, bias, lens, softplus, init,
                   dy, dfinal)
    close(out["y"], y.detach())
    close(out["final"], final.detach())
    for n_, t in grads.items():
        close(out[{"init": "dinit", "dt_bias": "ddt_bias"}.get(n_, "d" + n_)], t)
    # and against differences along one direction of all inputs
    dirs, eps = [normal(g, *t.shape) for t in plain], 1e-6
    with torch.no_grad():
        up, down = ([t + s * eps * d for t, d in zip(plain, dirs)] for s in (1, -1))
        (y1, f1), (y0, f0) = run(*up), run(*down)
    slope = float((((y1 - y0) * dy).sum() + ((f1 - f0) * dfinal).sum()) / (2 * eps))
    want = float(sum((grads[n_] * d).sum() for n_, d in zip(names, dirs)))
    assert abs(slope - want) <= 1e-6 * (1 + abs(want))


def test_quant():
    """Every code of a row, and halfway values to the even one."""
    codes = torch.tensor([448.0, 1.0, 1.0625, 1.1875, -0.0009765625, -0.0029296875, 0.0, 17.0])
    out = ref.quant(codes.double()[None], None, None, None, 1e-5, 8, ref.E4M3)
    want = codes.to(ref.E4M3).double()
    assert torch.equal(out["codes"][0], want)
    close(out["scales"] * out["codes"], out["scales"] * want)
