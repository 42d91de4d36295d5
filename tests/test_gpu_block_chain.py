"""The block operators together, as a block runs them: add norm, linear
attention, gated norm, add norm; forward and backward over packed prompts, then
single tokens from the prompts' states.  Everything in fp32 against the plain
forms in 64 bits.  Projections between them are a user's own and left out: the
normed stream is cut into q, k, v and the gate z directly.

Tolerance: each operator is good to some 2e-6 of its result (its own tests); a
chain of four, with norms that pass relative errors on unchanged and q, k, v
entering as products of three: 2e-6 * (1 + 3 + 1 + 1) * 3 < 5e-5 with the
gradients' chain of the same length on top.
"""
import pytest
import torch

import block_ref
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 5e-5
H, G, K, V = 4, 2, 64, 64
D = 2 * G * K + 2 * H * V


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


def split(y):
    """q, k [T, G, K], v [T, H, V] and z [T, H V] of the normed stream."""
    q, k, v, z = y.split([G * K, G * K, H * V, H * V], dim=-1)
    T = y.shape[0]
    return [t.contiguous() for t in (q.reshape(T, G, K), k.reshape(T, G, K), v.reshape(T, H, V), z)]


def close(name, got, ref):
    err = float((got.double().cpu() - ref).norm() / ref.norm())
    log(f"  {name}: {err:.2e}")
    assert err <= TOL, (name, err)


def test_block_forward_backward_and_steps(ssd):
    lens = [97, 1, 0, 200]
    T = sum(lens)
    g = torch.Generator().manual_seed(5)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    x, res = normal(T, D), normal(T, D)
    s, w, wv, w2 = normal(D), normal(D), normal(V), normal(H * V)
    ld = -torch.exp2(-torch.arange(1.0, H + 1))
    res2 = normal(T, H * V)
    dout, dh2 = normal(T, H * V), normal(T, H * V)
    cu = torch.tensor([0, 97, 98, 98, 298], dtype=torch.int32)

    # plain, 64 bits
    r1 = block_ref.add_norm(x.double(), res.double(), s.double(), w.double(), 1e-5)
    q, k, v, z = split(r1["y"])
    r2 = block_ref.linattn(q, k, v, ld, lens, K ** -0.5)
    o = r2["o"].reshape(T, H * V)
    r3 = block_ref.gated_norm(o, z, wv.double(), 1e-5, V, "silu", False)
    b4 = block_ref.add_norm(r3["y"], res2.double(), None, w2.double(), 1e-5, dout.double(),
                            dh2.double())
    b3 = block_ref.gated_norm(o, z, wv.double(), 1e-5, V, "silu", False, b4["dx"])
    b2 = block_ref.linattn(q, k, v, ld, lens, K ** -0.5, None, b3["dx"].reshape(T, H, V))
    dy = torch.cat([b2["dq"].reshape(T, -1), b2["dk"].reshape(T, -1), b2["dv"].reshape(T, -1),
                    b3["dz"]], dim=-1)
    b1 = block_ref.add_norm(x.double(), res.double(), s.double(), w.double(), 1e-5, dy)

    # the library
    x, res, s, w, wv, w2, ld, res2, dout, dh2, cu = (
        t.to(DEV) for t in (x, res, s, w, wv, w2, ld, res2, dout, dh2, cu))
    y, h = ssd.add_norm(x, res, s, w)
    gq, gk, gv, gz = split(y)
    a = (gq[None], gk[None], gv[None], ld)
    go, state = ssd.linattn(*a, None, cu)
    go = go.view(T, H * V)
    gy = ssd.gated_norm(go, gz, wv, group=V)
    y2, h2 = ssd.add_norm(gy, res2, None, w2)
    close("stream", h2, b4["h"])
    close("out", y2, b4["y"])
    close("state", state, r2["final"])
    dgy, dres2, _, dw2 = ssd.add_norm_backward(gy, res2, None, w2, dout, dh2)
    dgo, dgz, dwv = ssd.gated_norm_backward(go, gz, wv, dgy, group=V)
    dq, dk, dv, _ = ssd.linattn_backward(*a, dgo.view(1, T, H, V), None, None, cu)
    dyy = torch.cat([t.reshape(T, -1) for t in (dq, dk, dv)] + [dgz], dim=-1)
    dx, dres, ds, dw = ssd.add_norm_backward(x, res, s, w, dyy)
    for n, t, r in (("dx", dx, b1["dx"]), ("dresidual", dres, b1["dresidual"]),
                    ("dscale", ds, b1["dres_scale"]), ("dw", dw, b1["dweight"]),
                    ("dwv", dwv, b3["dweight"]), ("dw2", dw2, b4["dweight"]),
                    ("dresidual2", dres2, b4["dresidual"])):
        close(n, t, r)

    # one more token for every sequence, from the prompts' states
    n = len(lens)
    xt, rt = torch.randn(n, D, generator=g), torch.randn(n, D, generator=g)
    yt, _ = ssd.add_norm(xt.to(DEV), rt.to(DEV), s, w)
    tq, tk, tv, tz = split(yt)
    ot = torch.empty_like(tv)
    ssd.ssd_linattn_step(tq, tk, tv, ld, state, ot)
    out = ssd.gated_norm(ot.view(n, H * V), tz, wv, group=V)
    p1 = block_ref.add_norm(xt.double(), rt.double(), s.double().cpu(), w.double().cpu(), 1e-5)
    q, k, v, z = split(p1["y"])
    p2 = block_ref.linattn(q, k, v, ld.cpu(), [1] * n, K ** -0.5, r2["final"])
    p3 = block_ref.gated_norm(p2["o"].reshape(n, H * V), z, wv.double().cpu(), 1e-5, V, "silu",
                              False)
    close("next state", state, p2["final"])
    close("next out", out, p3["y"])
