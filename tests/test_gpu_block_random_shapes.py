"""The block operators over seeded draws of shapes, types, layouts and options, with
guard bytes around every output and workspace, which are as large as the calls ask for.

Linear attention: head by head, block_check.py has the tolerances.  Norms, on 2-norms:
2^-8 of a bf16 result for its own rounding, and for every result 2^-18 of the same
formula with each term's absolute value (a row's fp32 sums are over up to 16384 values
in 64 lanes or more, and the parameters' over up to 200 rows: sqrt(16384) / 4 + 16
roundings of 2^-24, the gate's exponential and reciprocal 2^-22)."""
import math
import random

import pytest
import torch

import block_ref
from block_check import check_heads, references
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
GUARD = 256
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


class Guarded:
    """Tensors with GUARD bytes of a pattern on either side; NaN bytes inside."""

    def __init__(self):
        self.buffers = []

    def __call__(self, shape, dtype):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
        buf[GUARD:GUARD + n] = 0xFF
        self.buffers.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        for buf, n in self.buffers:
            assert (buf[:GUARD] == 0xA5).all() and (buf[GUARD + n:] == 0xA5).all()


def spread(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw_linattn(i):
    rng = random.Random(9000 + i)
    G = rng.choice([1, 2, 3])
    c = {"i": i, "G": G, "H": G * rng.choice([1, 1, 2, 3]), "K": rng.choice([64, 128]),
         "V": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
         "init": rng.random() < 0.5, "dfinal": rng.random() < 0.5, "packed": rng.random() < 0.8,
         "in_place": rng.random() < 0.5}
    total = spread(rng, 1, 700)
    if c["packed"]:
        lens, left = [], total
        for _ in range(rng.choice([0, 1, 3, 9])):
            lens.append(rng.randint(0, left))
            left -= lens[-1]
        c |= {"lens": lens + [left], "before": rng.choice([0, 0, 3]),
              "after": rng.choice([0, 0, 70])}
    else:
        n = rng.choice([1, 2, 5])
        c |= {"lens": [max(1, total // n)] * n, "before": 0, "after": 0}
    return c


def name_of(c):
    return "_".join(f"{k[:2]}{v}" for k, v in c.items()).replace(" ", "")[:90]


@pytest.mark.parametrize("c", [draw_linattn(i) for i in range(28)], ids=name_of)
def test_linattn(ssd, c):
    log(f"[random] {c}")
    H, G, K, V, lens = (c[n] for n in ("H", "G", "K", "V", "lens"))
    dt, n, T = DTYPES[c["dtype"]], len(lens), sum(lens)
    g = torch.Generator().manual_seed(c["i"])
    rows, cut = T + c["before"] + c["after"], slice(c["before"], c["before"] + T)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g).to(dtype)

    s = {m: normal(rows, h, d, dtype=dt) for m, h, d in (("q", G, K), ("k", G, K), ("v", H, V),
                                                         ("do", H, V))}
    ld = -torch.exp(torch.empty(H).uniform_(-8, 2, generator=g))
    init = normal(n, H, K, V) if c["init"] else None
    dfinal = normal(n, H, K, V) if c["dfinal"] else None
    ref, size = references(*(s[m][cut] for m in ("q", "k", "v")), ld, lens, K ** -0.5, init,
                           s["do"][cut], dfinal)

    def dev(t):
        return None if t is None else t.to(DEV)

    cu = None
    if c["packed"]:
        cu = torch.tensor([c["before"] + sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32,
                          device=DEV)
    shape = (1, rows) if c["packed"] else (n, lens[0])
    q, k, v, do = (dev(s[m]).view(*shape, *s[m].shape[1:]) for m in ("q", "k", "v", "do"))
    out = Guarded()
    dims = ssd.LinattnDims(rows, n, H, G, K, V)
    results = []
    for _ in range(2):
        ws = [out((ssd.linattn_workspace_bytes(dims, dt, b),), torch.uint8) for b in (False, True)]
        o, dq, dk, dv = (out(t.shape, dt) for t in (v, q, k, v))
        final, dinit = (out((n, H, K, V), torch.float32) for _ in range(2))
        start = dev(init)
        if c["in_place"] and init is not None:
            final.copy_(start)
            start = final
        ssd.ssd_linattn_fwd(q, k, v, dev(ld), start, cu, o, final, ws[0])
        ssd.ssd_linattn_bwd(q, k, v, dev(ld), dev(init), cu, do, dev(dfinal), dq, dk, dv, dinit,
                            ws[1])
        results.append({"o": o, "dq": dq, "dk": dk, "dv": dv, "final": final, "dinit": dinit})
    out.check()
    got = {}
    for m, t in results[0].items():
        assert torch.equal(t.contiguous().view(torch.uint8),
                           results[1][m].contiguous().view(torch.uint8)), m
        if m in ("final", "dinit"):
            got[m] = t
        else:
            t = t.reshape(rows, *t.shape[2:])
            assert torch.isnan(torch.cat([t[:cut.start], t[cut.stop:]])).all(), m   # left alone
            got[m] = t[cut]
    worst = check_heads(got, ref, size, T)
    log("  of the tolerance " + ", ".join(f"{m} {w:.2f}" for m, w in worst.items()))


def close(name, got, ref, size):
    g = got.double().cpu()
    assert g.shape == ref.shape and torch.isfinite(g).all(), name
    tol = 2.0 ** -18 * float(size.norm())
    if got.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * float(ref.norm())
    err = float((g - ref).norm())
    log(f"  {name}: {err / max(tol, 1e-300):.2f} of the tolerance")
    assert err <= tol, (name, err, tol)


def draw_norm(i):
    rng = random.Random(7000 + i)
    c = {"i": i, "op": "add" if i % 2 else "gate", "rows": spread(rng, 1, 200),
         "xt": rng.choice(["bf16", "fp32"]), "rt": rng.choice(["bf16", "fp32"]),
         "weight": rng.random() < 0.8}
    if c["op"] == "add":
        return c | {"dim": spread(rng, 16, 16384), "residual": rng.random() < 0.8,
                    "scale": rng.random() < 0.5, "dh": rng.random() < 0.7}
    group = spread(rng, 16, 16384)
    per = rng.choice([1, 2, 5, 20, 33]) if group < 300 else rng.choice([1, 2])
    return c | {"group": group, "dim": group * per, "gate": rng.choice(["silu", "sigmoid"]),
                "first": rng.random() < 0.5, "z": rng.random() < 0.9,
                "shared": rng.random() < 0.5}


@pytest.mark.parametrize("c", [draw_norm(i) for i in range(48)], ids=name_of)
def test_norms(ssd, c):
    log(f"[random] {c}")
    g = torch.Generator().manual_seed(c["i"])
    rows, D, dt, rdt = c["rows"], c["dim"], DTYPES[c["xt"]], DTYPES[c["rt"]]

    def normal(*shape, dtype=torch.float32, there=True):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV) if there else None

    def dbl(t):
        return None if t is None else t.double().cpu()

    out = Guarded()
    x = normal(rows, D, dtype=dt)
    if c["op"] == "add":
        res = normal(rows, D, dtype=rdt, there=c["residual"])
        rdt = rdt if c["residual"] else dt
        s, w = normal(D, there=c["scale"]), normal(D, there=c["weight"])
        dy, dh = normal(rows, D, dtype=dt), normal(rows, D, dtype=rdt, there=c["dh"])
        y, h, dx = out((rows, D), dt), out((rows, D), rdt), out((rows, D), dt)
        dres = out((rows, D), rdt) if c["residual"] else None
        ds, dw = (out((D,), torch.float32) if t is not None else None for t in (s, w))
        ws = out((ssd.add_norm_workspace_bytes(rows, D),), torch.uint8)
        ssd.ssd_add_norm_fwd(x, res, s, w, y, h, EPS)
        ssd.ssd_add_norm_bwd(x, res, s, w, dy, dh, dx, dres, ds, dw, ws, EPS)
        out.check()
        xd, rd, sd, wd, dyd, dhd = (dbl(t) for t in (x, res, s, w, dy, dh))
        ref = block_ref.add_norm(xd, rd, sd, wd, EPS, dyd, dhd)
        sd, wd = (torch.ones(D).double() if t is None else t.abs() for t in (sd, wd))
        ha = (xd.abs() * sd) + (0 if rd is None else rd.abs())
        r = 1 / torch.sqrt((ref["h"] ** 2).mean(-1, keepdim=True) + EPS)
        n, e = ha * r, dyd.abs() * wd
        ga = r * (e + n * (e * n).mean(-1, keepdim=True)) + (0 if dhd is None else dhd.abs())
        size = {"y": n * wd, "h": ha, "dx": ga * sd, "dresidual": ga,
                "dres_scale": (ga * xd.abs()).sum(0), "dweight": (dyd.abs() * n).sum(0)}
        got = {"y": y, "h": h, "dx": dx, "dresidual": dres, "dres_scale": ds, "dweight": dw}
    else:
        group, first = c["group"], c["first"]
        z = normal(rows, D, dtype=rdt, there=c["z"])
        wdim = group if c["shared"] else D
        w = normal(wdim, there=c["weight"])
        dy = normal(rows, D, dtype=rdt)
        y, dx = out((rows, D), rdt), out((rows, D), dt)
        dz = out((rows, D), rdt) if c["z"] else None
        dw = out((wdim,), torch.float32) if c["weight"] else None
        dims = ssd.GatedNormDims(rows, D, group, wdim if c["weight"] else D)
        ws = out((ssd.gated_norm_workspace_bytes(dims),), torch.uint8)
        ssd.ssd_gated_norm_fwd(x, z, w, y, EPS, group, c["gate"], first)
        ssd.ssd_gated_norm_bwd(x, z, w, dy, dx, dz, dw, ws, EPS, group, c["gate"], first)
        out.check()
        xd, zd, wd, dyd = (dbl(t) for t in (x, z, w, dy))
        ref = block_ref.gated_norm(xd, zd, wd, EPS, group, c["gate"], first, dyd)
        x3, d3 = xd.view(rows, -1, group), dyd.abs().view(rows, -1, group)
        w3 = torch.ones(1, group).double() if wd is None else wd.abs().view(-1, group)
        act, dact = torch.ones_like(x3), torch.zeros_like(x3)
        if zd is not None:
            z3 = zd.view_as(x3)
            sig = torch.sigmoid(z3)
            dsig = sig * (1 - sig)
            act, dact = ((z3.abs() * sig, sig + z3.abs() * dsig) if c["gate"] == "silu"
                         else (sig, dsig))
        u = x3.abs() * act if first else x3.abs()
        r = 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS)
        n, dn = u * r, d3 if first else d3 * act
        e = dn * w3
        du = r * (e + n * (e * n).mean(-1, keepdim=True))
        size = {"y": n * w3 * (1 if first else act), "dx": du * act if first else du,
                "dz": (du * x3.abs() if first else d3 * n * w3) * dact}
        size = {m: t.reshape(rows, D) for m, t in size.items()}
        dws = (dn * n).sum(0)
        size["dweight"] = dws.sum(0) if c["shared"] else dws.reshape(-1)
        if c["shared"] and group == D:
            size["dweight"] = dws.reshape(-1)
        got = {"y": y, "dx": dx, "dz": dz, "dweight": dw}
    for m, t in got.items():
        if t is not None:
            close(m, t, ref[m].reshape(t.shape), size[m].reshape(t.shape))


@pytest.mark.parametrize("i", range(12))
def test_linattn_step(ssd, i):
    rng = random.Random(5000 + i)
    G = rng.choice([1, 2, 5, 8])
    b, H, K, V = spread(rng, 1, 90), G * rng.choice([1, 3]), *rng.choices([64, 128], k=2)
    dtype = rng.choice(["bf16", "fp32"])
    log(f"[random] step b={b} H={H} G={G} K={K} V={V} {dtype}")
    g = torch.Generator().manual_seed(i)
    dt, out = DTYPES[dtype], Guarded()
    q, k, v = (torch.randn(b, h, d, generator=g).to(dt) for h, d in ((G, K), (G, K), (H, V)))
    init, ld = torch.randn(b, H, K, V, generator=g), -torch.rand(H, generator=g)
    o, state = out((b, H, V), dt), out((b, H, K, V), torch.float32)
    state.copy_(init)
    ssd.ssd_linattn_step(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), state, o)
    out.check()
    ref, size = references(q, k, v, ld, [1] * b, K ** -0.5, init)
    check_heads({"o": o, "final": state}, ref, size, b)
