"""The operators of a block with a selective state space run together, as a block runs
them: norm (also in 8 bits), short convolution, scan with its gate, forward and backward over
packed prompts, then single tokens from the prompts' states; captured in a HIP graph;
and on a stream of their own.  In fp32 against the plain forms in 64 bits.  Projections
between them are a user's own: the normed stream is cut into x and z, and the convolution's
result into what the scan takes.

Tolerance: each operator is good to some 2e-6 of its result (its own tests); a chain of three,
forward and backward, with products of up to three computed factors: 2e-6 * 3 * 2 * 3 < 5e-5.
"""
import pytest
import torch

import block_ref
import selective_ref as ref
from gpu_util import log
from selective_util import same_bits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 5e-5
D, N, W = 64, 16, 4
E = 2 * D + 2 * N           # x, z, B and C of the normed stream
LENS = [97, 1, 0, 200]


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


def close(name, got, want):
    err = float((got.double().cpu() - want).norm() / want.norm())
    log(f"  {name}: {err:.2e}")
    assert err <= TOL, (name, err)


def inputs(seed=3):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    T, n = sum(LENS), len(LENS)
    return {"x": normal(T, E), "res": normal(T, E), "w": normal(E) * 0.3 + 1,
            "cw": normal(D, W) * 0.5, "cb": normal(D) * 0.1, "A": -torch.rand(D, N, generator=g) * N,
            "Dk": normal(D), "bias": normal(D) * 0.5 - 2, "cinit": normal(n, W - 1, D),
            "sinit": normal(n, D, N), "dy": normal(T, D), "x1": normal(n, E), "r1": normal(n, E)}


def cut(y):
    """x, z, B, C: columns of the normed stream, as a projection would give them."""
    return y[..., :D], y[..., D:2 * D], y[..., 2 * D:2 * D + N], y[..., 2 * D + N:]


def device(t):
    return {k: v.to(DEV) for k, v in t.items()}


CU = [0, 97, 98, 98, 298]


def forward(ssd, t, cu):
    y, h = ssd.add_norm(t["x"], t["res"], None, t["w"])
    x, z, B, C = cut(y[None])
    c, cstate = ssd.short_conv(x, t["cw"], t["cb"], t["cinit"], cu)
    a = (c, x, t["A"], B.unflatten(-1, (1, N)), C.unflatten(-1, (1, N)), t["Dk"], z, t["bias"])
    o, sstate = ssd.selective_scan(*a, t["sinit"], cu)
    return y, x, a, o, cstate, sstate


def backward(ssd, t, cu, x, a):
    g = ssd.selective_scan_backward(*a, t["dy"][None], None, t["sinit"], cu)
    dc, ddt, dA, dB, dC, dD, dz, dbias, dsinit = g
    dx, dcw, dcb, dcinit = ssd.short_conv_backward(x, t["cw"], t["cb"], dc, None, t["cinit"], cu)
    dyn = torch.cat([dx + ddt, dz, dB.flatten(2), dC.flatten(2)], -1)[0]
    dxx, dres, _, dw = ssd.add_norm_backward(t["x"], t["res"], None, t["w"], dyn)
    return {"dx": dxx, "dw": dw, "dcw": dcw, "dcb": dcb, "dA": dA, "dD": dD, "dbias": dbias,
            "dcinit": dcinit, "dsinit": dsinit}


def test_block_forward_backward_and_steps(ssd):
    t = inputs()
    d = {k: v.double() for k, v in t.items()}
    r1 = block_ref.add_norm(d["x"], d["res"], None, d["w"], 1e-5)
    x, z, B, C = cut(r1["y"])
    r2 = ref.conv(x, d["cw"], d["cb"], LENS, True, d["cinit"])
    scan = (r2["y"], x, d["A"], B[:, None], C[:, None], d["Dk"], z, d["bias"], LENS, True,
            d["sinit"])
    r3 = ref.scan(*scan, d["dy"])
    b2 = ref.conv(x, d["cw"], d["cb"], LENS, True, d["cinit"], r3["dx"])
    dyn = torch.cat([b2["dx"] + r3["ddt"], r3["dz"], r3["dB"][:, 0], r3["dC"][:, 0]], -1)
    b1 = block_ref.add_norm(d["x"], d["res"], None, d["w"], 1e-5, dyn)
    want = {"dx": b1["dx"], "dw": b1["dweight"], "dcw": b2["dweight"], "dcb": b2["dbias"],
            "dA": r3["dA"], "dD": r3["dD"], "dbias": r3["ddt_bias"], "dcinit": b2["dinit"],
            "dsinit": r3["dinit"]}

    t = device(t)
    cu = torch.tensor(CU, dtype=torch.int32, device=DEV)
    _, gx, a, o, cstate, sstate = forward(ssd, t, cu)
    close("out", o[0], r3["y"])
    close("conv state", cstate, r2["final"])
    close("scan state", sstate, r3["final"])
    for n, v in backward(ssd, t, cu, gx, a).items():
        close(n, v, want[n])

    # one more token for every sequence, from the prompts' states
    y1, _ = ssd.add_norm(t["x1"], t["r1"], None, t["w"])
    x1, z1, B1, C1 = cut(y1)
    c1, o1 = torch.empty(4, D, device=DEV), torch.empty(4, D, device=DEV)
    ssd.ssd_short_conv_step(x1, t["cw"], t["cb"], cstate, c1)
    ssd.ssd_selective_scan_step(c1, x1, t["A"], B1.unflatten(-1, (1, N)), C1.unflatten(-1, (1, N)),
                                t["Dk"], z1, t["bias"], sstate, o1)
    p1 = block_ref.add_norm(d["x1"], d["r1"], None, d["w"], 1e-5)
    x, z, B, C = cut(p1["y"])
    p2 = ref.conv(x, d["cw"], d["cb"], [1] * 4, True, r2["final"])
    p3 = ref.scan(p2["y"], x, d["A"], B[:, None], C[:, None], d["Dk"], z, d["bias"], [1] * 4,
                  True, r3["final"])
    close("next out", o1, p3["y"])
    close("next conv state", cstate, p2["final"])
    close("next scan state", sstate, p3["final"])

    # the same norm for a projection in 8 bits: half a step of 2^-4 of the group's scale
    codes, scales, h8 = ssd.add_norm_quant(t["x1"], t["r1"], None, t["w"])
    err = (codes.float() * scales - y1).abs()
    assert (err <= y1.abs() * 2.0 ** -4 * 1.01 + scales * 2.0 ** -10).all()
    assert same_bits(h8, ssd.add_norm(t["x1"], t["r1"], None, t["w"])[1])


def test_block_from_a_graph(ssd):
    """Forward, backward, 8-bit norm and a step captured once and replayed, with eager work of
    the same calls in between; every replay gives the eager bits."""
    t = device(inputs(4))
    cu = torch.tensor(CU, dtype=torch.int32, device=DEV)
    states = [torch.zeros(4, W - 1, D, device=DEV), torch.zeros(4, D, N, device=DEV)]

    def run():
        y, x, a, o, cstate, sstate = forward(ssd, t, cu)
        g = backward(ssd, t, cu, x, a)
        codes, scales, _ = ssd.add_norm_quant(t["x"], t["res"], None, t["w"])
        x1, z1, B1, C1 = cut(y[:4])
        c1, o1 = torch.empty(4, D, device=DEV), torch.empty(4, D, device=DEV)
        states[0].copy_(cstate)
        states[1].copy_(sstate)
        ssd.ssd_short_conv_step(x1, t["cw"], t["cb"], states[0], c1)
        ssd.ssd_selective_scan_step(c1, x1, t["A"], B1.unflatten(-1, (1, N)),
                                    C1.unflatten(-1, (1, N)), t["Dk"], z1, t["bias"], states[1],
                                    o1)
        return [o, cstate, sstate, *g.values(), codes, scales, c1, o1]

    want = [v.clone() for v in run()]
    last = [s.clone() for s in states]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    torch.cuda.synchronize()
    for rep in range(3):
        for v in got:
            v.view(torch.uint8).fill_(0xFF)
        for s in states:
            s.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + states, want + last):
            assert same_bits(a, b), rep
        for a, b in zip(run(), want):        # eager work between replays
            assert same_bits(a, b), rep


def test_two_streams_at_once(ssd):
    cu = torch.tensor(CU, dtype=torch.int32, device=DEV)
    ts = [device(inputs(s)) for s in (5, 6)]
    want = []
    for t in ts:
        _, x, a, o, c, s = forward(ssd, t, cu)
        want.append([o, c, s, *backward(ssd, t, cu, x, a).values()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = [None, None]
    for rep in range(3):
        for i, (t, st) in enumerate(zip(ts, streams)):
            with torch.cuda.stream(st):
                _, x, a, o, c, s = forward(ssd, t, cu)
                got[i] = [o, c, s, *backward(ssd, t, cu, x, a).values()]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(same_bits(a, b) for a, b in zip(g, w)), rep


def test_inside_an_autograd_function(ssd):
    """A user's own functions around the pairs: their gradients are those of the calls."""
    class Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            ctx.save_for_backward(x, w, b)
            return ssd.short_conv(x, w, b)[0]

        @staticmethod
        def backward(ctx, dy):
            return ssd.short_conv_backward(*ctx.saved_tensors, dy.contiguous())[:3]

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *a):
            ctx.save_for_backward(*a)
            return ssd.selective_scan(*a)[0]

        @staticmethod
        def backward(ctx, dy):
            return ssd.selective_scan_backward(*ctx.saved_tensors, dy.contiguous())[:8]

    t = device(inputs(7))
    y = t["x"][None].clone()
    leaves = [v.requires_grad_() for v in (y, t["cw"], t["cb"], t["A"], t["Dk"], t["bias"])]
    x, z, B, C = cut(y)
    o = Scan.apply(Conv.apply(x, t["cw"], t["cb"]), x, t["A"], B.unflatten(-1, (1, N)),
                   C.unflatten(-1, (1, N)), t["Dk"], z, t["bias"])
    o.backward(t["dy"][None])
    with torch.no_grad():
        c, _ = ssd.short_conv(x, t["cw"], t["cb"])
        g = ssd.selective_scan_backward(c, x, t["A"], B.unflatten(-1, (1, N)),
                                        C.unflatten(-1, (1, N)), t["Dk"], z, t["bias"],
                                        t["dy"][None])
        dx, dcw, dcb, _ = ssd.short_conv_backward(x, t["cw"], t["cb"], g[0])
        dy = torch.cat([dx + g[1], g[6], g[3].flatten(2), g[4].flatten(2)], -1)
    for leaf, w in zip(leaves, (dy, dcw, dcb, g[2], g[5], g[7])):
        assert float((leaf.grad - w).norm()) <= 1e-6 * float(w.norm())
