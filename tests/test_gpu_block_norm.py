"""The norms around a block (ssd_add_norm_fwd, _bwd and ssd_gated_norm_fwd, _bwd)
against plain forms in 64 bits.

Tolerances, on the 2-norm of the difference over that of the result: a tensor
stored in bf16 is rounded once, by 2^-8 of the value at most; one in fp32 is
the result of a few dozen fp32 operations of 2^-24 each (the gate's exponential
and reciprocal are good to 2^-22) and of sums whose roundings grow like the
square root of their length over the row of up to 5120: 2^-24 sqrt(5120) / 4
(partial sums are held by 64 lanes or more) + 16 * 2^-24 < 34 * 2^-24 = 2e-6.
The gradients of weights and scales are fp32 sums over the rows: the same.
"""
import pytest
import torch

import block_ref
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 2e-6}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


def check(name, got, ref):
    g = got.double().cpu()
    assert g.shape == ref.shape and torch.isfinite(g).all(), name
    norm = float(ref.norm())
    err = float((g - ref).norm()) / norm if norm else float(g.abs().max())
    log(f"  {name}: {err:.2e} (at most {TOL[got.dtype]:.2e})")
    assert err <= TOL[got.dtype], (name, err)


def dbl(t):
    return None if t is None else t.double().cpu()


ADD_CASES = [
    # rows, dim, x, residual's type (None: no residual), scale, weight, dh
    (1, 1, "fp32", "fp32", True, True, True),
    (3, 33, "bf16", "fp32", True, True, True),
    (5, 64, "bf16", "bf16", False, True, True),
    (2, 250, "fp32", "bf16", True, False, False),
    (300, 768, "bf16", "bf16", True, True, True),
    (7, 1001, "bf16", "bf16", False, False, True),
    (33, 2560, "bf16", "fp32", True, True, True),
    (2049, 520, "bf16", "fp32", True, True, True),    # more rows than teams
    (9, 2051, "fp32", "fp32", True, True, True),
    (3, 4104, "fp32", "fp32", True, True, False),
    (4, 5119, "bf16", "bf16", True, True, True),
    (2, 16384, "bf16", "fp32", True, True, True),
    (3, 8200, "bf16", "bf16", True, True, True),
    (3, 16383, "bf16", "fp32", True, True, True),
    (4, 128, "bf16", None, True, True, True),
    (4, 128, "fp32", None, False, True, False),
]


@pytest.mark.parametrize("rows,dim,xt,rt,scaled,weighted,dhs", ADD_CASES,
                         ids=lambda v: str(v))
def test_add_norm(ssd, rows, dim, xt, rt, scaled, weighted, dhs):
    g = torch.Generator().manual_seed(rows * dim)
    dt, rdt = DTYPES[xt], DTYPES[rt or xt]
    log(f"[add_norm] {rows}x{dim} {xt} {rt}")

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV)

    x, dy = normal(rows, dim, dtype=dt), normal(rows, dim, dtype=dt)
    res = normal(rows, dim, dtype=rdt) if rt else None
    dh = normal(rows, dim, dtype=rdt) if dhs else None
    s, w = (normal(dim) if scaled else None), (normal(dim) if weighted else None)
    y, h = ssd.add_norm(x, res, s, w, EPS)
    ref = block_ref.add_norm(dbl(x), dbl(res), dbl(s), dbl(w), EPS, dbl(dy), dbl(dh))
    check("y", y, ref["y"])
    check("h", h, ref["h"])
    dx, dres, ds, dw = ssd.add_norm_backward(x, res, s, w, dy, dh, EPS)
    check("dx", dx, ref["dx"])
    for n, t, there in (("dresidual", dres, res), ("dres_scale", ds, s), ("dweight", dw, w)):
        assert (t is None) == (there is None)
        if t is not None:
            check(n, t, ref[n])


GATE_CASES = [
    # rows, dim, group, weight, x, z, gate, first, with z
    (1, 64, 64, "dim", "bf16", "bf16", "silu", False, True),
    (3, 33, 33, "dim", "fp32", "bf16", "silu", True, True),
    (130, 320, 64, "group", "bf16", "bf16", "silu", False, True),
    (65, 384, 128, "group", "fp32", "bf16", "silu", True, True),
    (17, 1280, 256, "dim", "bf16", "fp32", "sigmoid", False, True),
    (700, 1536, 1536, "dim", "fp32", "bf16", "silu", True, True),
    (5, 99, 33, "group", "bf16", "bf16", "sigmoid", True, True),
    (4, 5120, 2560, "dim", "bf16", "bf16", "silu", True, True),
    (3, 300, 300, "dim", "fp32", "fp32", "sigmoid", False, True),
    (2, 1500, 750, "group", "bf16", "bf16", "silu", False, True),
    (6, 256, 64, "none", "fp32", "fp32", "silu", True, True),
    (40, 512, 128, "dim", "bf16", "bf16", "silu", False, False),
    (40, 512, 128, "group", "fp32", "fp32", "silu", True, False),
    (2100, 40, 8, "dim", "bf16", "bf16", "silu", True, True),
    (33, 30, 3, "group", "bf16", "bf16", "silu", False, True),      # less than a vector
    (33, 77, 11, "dim", "bf16", "fp32", "silu", True, True),        # vectors that overlap
    (5, 9000, 9000, "dim", "bf16", "bf16", "silu", True, True),
    (5, 8193, 8193, "dim", "fp32", "bf16", "sigmoid", False, True),
]


@pytest.mark.parametrize("rows,dim,group,wt,xt,zt,gate,first,gated", GATE_CASES,
                         ids=lambda v: str(v))
def test_gated_norm(ssd, rows, dim, group, wt, xt, zt, gate, first, gated):
    g = torch.Generator().manual_seed(rows * dim + group)
    dt, zdt = DTYPES[xt], DTYPES[zt if gated else xt]
    log(f"[gated_norm] {rows}x{dim} by {group} {xt} {zt} {gate} first={first}")

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV)

    x, dy = normal(rows, dim, dtype=dt), normal(rows, dim, dtype=zdt)
    z = normal(rows, dim, dtype=zdt) if gated else None
    w = None if wt == "none" else normal(dim if wt == "dim" else group)
    y = ssd.gated_norm(x, z, w, EPS, group, gate, first)
    ref = block_ref.gated_norm(dbl(x), dbl(z), dbl(w), EPS, group, gate, first, dbl(dy))
    check("y", y, ref["y"])
    dx, dz, dw = ssd.gated_norm_backward(x, z, w, dy, EPS, group, gate, first)
    check("dx", dx, ref["dx"])
    assert (dz is None) == (z is None) and (dw is None) == (w is None)
    if dz is not None:
        check("dz", dz, ref["dz"])
    if dw is not None:
        check("dweight", dw, ref["dweight"])


def test_far_gates_and_empty_rows(ssd):
    """Gates far out (sigmoid 0 or 1, act 0 or z) and rows of zeros: finite
    values, and what the formulas give."""
    x = torch.randn(6, 128, generator=torch.Generator().manual_seed(3)).to(DEV)
    z = torch.tensor([-1e4, -90.0, -20.0, 20.0, 90.0, 1e4]).repeat(22)[:128].to(DEV).expand(6, 128)
    z = z.contiguous()
    x[2] = 0.0
    dy = torch.ones_like(x)
    for gate in ("silu", "sigmoid"):
        for first in (False, True):
            zz = z.clamp(-1e4, 30.0) if first and gate == "silu" else z
            ref = block_ref.gated_norm(dbl(x), dbl(zz), None, EPS, 64, gate, first, dbl(dy))
            check("y", ssd.gated_norm(x, zz, None, EPS, 64, gate, first), ref["y"])
            dx, dz, _ = ssd.gated_norm_backward(x, zz, None, dy, EPS, 64, gate, first)
            check("dx", dx, ref["dx"])
            check("dz", dz, ref["dz"])
    zero = torch.zeros(3, 64, device=DEV)
    y, h = ssd.add_norm(zero, zero)
    assert not y.any() and not h.any()


def test_a_row_of_nan_stays_alone(ssd):
    x = torch.randn(9, 512, generator=torch.Generator().manual_seed(4)).to(DEV)
    want_y, want_h = ssd.add_norm(x, x)
    bad = x.clone()
    bad[4] = float("nan")
    y, h = ssd.add_norm(bad, bad)
    keep = torch.tensor([0, 1, 2, 3, 5, 6, 7, 8], device=DEV)
    assert torch.equal(y[keep], want_y[keep]) and torch.equal(h[keep], want_h[keep])
    assert torch.isnan(y[4]).all()


@pytest.mark.parametrize("dim", [768, 771, 4999])
def test_in_place(ssd, dim):
    g = torch.Generator().manual_seed(6)
    x, r, dy, dh = (torch.randn(50, dim, generator=g).to(torch.bfloat16).to(DEV) for _ in range(4))
    w = torch.randn(dim, generator=g).to(DEV)
    y, h = ssd.add_norm(x, r, None, w)
    x2, r2 = x.clone(), r.clone()
    ssd.ssd_add_norm_fwd(x2, r2, None, w, x2, r2)
    assert torch.equal(x2, y) and torch.equal(r2, h)
    dx, dres, _, dw = ssd.add_norm_backward(x, r, None, w, dy, dh)
    dy2, dh2, dw2 = dy.clone(), dh.clone(), torch.empty_like(w)
    ws = torch.empty(ssd.add_norm_workspace_bytes(50, dim), dtype=torch.uint8, device=DEV)
    ssd.ssd_add_norm_bwd(x, r, None, w, dy2, dh2, dy2, dh2, None, dw2, ws)
    assert torch.equal(dy2, dx) and torch.equal(dh2, dres) and torch.equal(dw2, dw)
    y = ssd.gated_norm(x, r, w)
    for into in (x.clone(), r.clone()):
        a, b = (into, r) if torch.equal(into, x) else (x, into)
        ssd.ssd_gated_norm_fwd(a, b, w, into)
        assert torch.equal(into, y)
    dx, dz, dw = ssd.gated_norm_backward(x, r, w, dy)
    dy2 = dy.clone()
    dx2 = torch.empty_like(x)
    d = ssd.GatedNormDims(50, dim, dim, dim)
    ws = torch.empty(ssd.gated_norm_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    ssd.ssd_gated_norm_bwd(x, r, w, dy2, dx2, dy2, dw2, ws)
    assert torch.equal(dy2, dz) and torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_gradients_against_differences(ssd):
    """Central differences of the fp32 forward calls: with a step of 1e-2 the
    next term of the series is below 1e-4 of the first for values of size 1,
    and the fp32 rounding of sums over 3e3 outputs, divided by the step, below
    2^-24 * 3e3 / 2e-2 ~ 1e-2 of one output: 1e-3 of the gradient's norm."""
    g = torch.Generator().manual_seed(8)
    x, z, dy, dh = (torch.randn(4, 192, generator=g).to(DEV) for _ in range(4))
    w, s = torch.randn(192, generator=g).to(DEV), torch.randn(192, generator=g).to(DEV)

    def add(t):
        y, h = ssd.add_norm(t["x"], t["z"], t["s"], t["w"], EPS)
        return float((y.double() * dy).sum() + (h.double() * dh).sum())

    def gated(t):
        return float((ssd.gated_norm(t["x"], t["z"], t["w"], EPS, 64, "silu", t["first"]).double()
                      * dy).sum())

    base = {"x": x, "z": z, "w": w, "s": s, "first": True}
    runs = [(add, base, dict(zip("xzsw", ssd.add_norm_backward(x, z, s, w, dy, dh, EPS))))]
    for first in (True, False):
        grads = ssd.gated_norm_backward(x, z, w, dy, EPS, 64, "silu", first)
        runs.append((gated, dict(base, first=first), dict(zip("xzw", grads))))
    for f, at, grads in runs:
        for n, grad in grads.items():
            step = torch.randn(at[n].shape, generator=g).to(DEV)
            up, down = (f(dict(at, **{n: at[n] + d * step})) for d in (1e-2, -1e-2))
            want = float((grad.double() * step.double()).sum())
            size = float(grad.double().norm())
            log(f"  {f.__name__} {n}: difference {(up - down) / 2e-2:.4f} gradient {want:.4f}")
            assert abs((up - down) / 2e-2 - want) <= 1e-3 * size * 3


def test_captured_and_replayed(ssd):
    g = torch.Generator().manual_seed(10)
    x, z, dy = (torch.randn(300, 640, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3))
    w = torch.randn(64, generator=g).to(DEV)
    wd = torch.randn(640, generator=g).to(DEV)

    def go():
        y, h = ssd.add_norm(x, z, wd, wd)
        return [y, h, *ssd.add_norm_backward(x, z, wd, wd, dy, dy),
                ssd.gated_norm(x, z, w, 1e-5, 64),
                *ssd.gated_norm_backward(x, z, w, dy, 1e-5, 64)]

    want = [t.clone() for t in go()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        assert torch.equal(ssd.add_norm(x, z, wd, wd)[0], want[0])


def test_refusals(ssd):
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, device=DEV)
    with pytest.raises(ValueError):
        ssd.add_norm(x, x[:2])
    with pytest.raises(TypeError):
        ssd.add_norm(x, None, None, w.to(torch.bfloat16))
    with pytest.raises(ValueError):
        ssd.add_norm(x.t(), None)
    with pytest.raises(ssd.SsdError):
        ssd.add_norm(x, None, None, w, 0.0)
    with pytest.raises(ValueError):
        ssd.gated_norm(x, x, w[:32], group=64)
    with pytest.raises(ssd.SsdError):
        ssd.gated_norm(x, x, None, group=48)
    with pytest.raises(ValueError):
        ssd.gated_norm(x, x, w, gate="relu")
    with pytest.raises(TypeError):
        ssd.gated_norm(x, x.half(), w)
    ws = torch.empty(16, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        ssd.ssd_gated_norm_bwd(x, x, w, x, torch.empty_like(x), None, None, ws)
    with pytest.raises(ssd.SsdError) as e:
        ssd.ssd_add_norm_bwd(x, None, None, w, x, None, torch.empty_like(x), None, None,
                             torch.empty_like(w), ws)
    assert e.value.status == ssd.SSD_ERR_WORKSPACE


def test_offsets_past_32_bits(ssd):
    """More than 2^31 elements, equal rows: the last has the first one's results."""
    rows, dim, group = 70000, 31000, 248
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(1, dim, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(dim, generator=g, device=DEV)
    want = ssd.gated_norm(x, x, w, EPS, group)
    want_dx, want_dz, _ = ssd.gated_norm_backward(x, x, w, x, EPS, group)
    x = x.expand(rows, dim).contiguous()
    assert x.numel() > 2 ** 31
    y = ssd.gated_norm(x, x, w, EPS, group)
    assert torch.equal(y[:1], want) and torch.equal(y[-1:], want)
    dx, dz, _ = ssd.gated_norm_backward(x, x, w, x, EPS, group)
    for t, r in ((dx, want_dx), (dz, want_dz)):
        assert torch.equal(t[:1], r) and torch.equal(t[-1:], r)
