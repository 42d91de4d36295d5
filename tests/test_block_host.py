"""Host-side checks of the block operators' C ABI (no GPU needed).

As in test_abi_host.py: every call below fails argument validation, which the
library performs on the host before any HIP call, so nothing is launched and
no pointer is touched; the module refuses to run where a GPU is visible.
"""
import ctypes
import subprocess

import pytest
import torch

if torch.cuda.is_available():
    pytest.skip("host-only validation tests use fake device pointers; "
                "not run where a GPU is visible", allow_module_level=True)

import mamba_ssd_chunked_fwd_amd as ssd  # noqa: E402

INV, UNS, WS = (ssd.SSD_ERR_INVALID_ARGUMENT, ssd.SSD_ERR_UNSUPPORTED, ssd.SSD_ERR_WORKSPACE)
lib = ssd.library()
FAKE = ctypes.c_void_p(0x7F0000000000)       # 16-byte aligned, never used
MISALIGNED = ctypes.c_void_p(0x7F0000000004)
ODD = ctypes.c_void_p(0x7F0000000002)


def test_every_declared_function_is_exported():
    names = ssd.header_functions(ssd.BLOCK_HEADER_PATH)
    assert len(names) == len(set(names)) == 11
    out = subprocess.run(["nm", "-D", "--defined-only", ssd.LIB_PATH],
                         capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    for n in names:
        assert n in exported, n


def ldims(**kw):
    base = dict(tokens=512, nseq=2, nheads=4, ngroups=2, dk=128, dv=64)
    base.update(kw)
    return ssd.LinattnDims(**base)


def _ref(d):
    return None if d is None else ctypes.byref(d)


def fwd(d, **o):
    return lib.ssd_linattn_fwd(
        o.get("q", FAKE), o.get("k", FAKE), o.get("v", FAKE), o.get("ld", FAKE),
        o.get("init"), o.get("cu"), o.get("out", FAKE), o.get("fin"), o.get("ws", FAKE),
        o.get("wsb", 1 << 40), 1.0, o.get("dt", ssd.SSD_BF16), _ref(d), None)


def bwd(d, **o):
    return lib.ssd_linattn_bwd(
        o.get("q", FAKE), o.get("k", FAKE), o.get("v", FAKE), o.get("ld", FAKE),
        o.get("init"), o.get("cu"), o.get("do", FAKE), o.get("dfin"), o.get("dq", FAKE),
        o.get("dk", FAKE), o.get("dv", FAKE), o.get("dinit"), o.get("ws", FAKE),
        o.get("wsb", 1 << 40), 1.0, o.get("dt", ssd.SSD_BF16), _ref(d), None)


def step(d, **o):
    return lib.ssd_linattn_step(
        o.get("q", FAKE), o.get("k", FAKE), o.get("v", FAKE), o.get("ld", FAKE),
        o.get("state", FAKE), o.get("out", FAKE), 1.0, o.get("dt", ssd.SSD_BF16), _ref(d), None)


BAD_DIMS = [
    (dict(tokens=0), INV), (dict(tokens=1 << 31), INV), (dict(nheads=0), INV),
    (dict(ngroups=3), INV), (dict(ngroups=0), INV), (dict(ngroups=8), INV),
    (dict(dk=96), UNS), (dict(dv=256), UNS), (dict(dk=-64), INV),
    (dict(nheads=1 << 16, ngroups=1), UNS), (dict(tokens=1 << 30), UNS),
]


@pytest.mark.parametrize("kw,expect", BAD_DIMS)
def test_linattn_rejects_bad_dims(kw, expect):
    d = ldims(**kw)
    assert fwd(d) == expect and bwd(d) == expect and step(d) == expect
    assert lib.ssd_linattn_fwd_workspace_bytes(_ref(d), ssd.SSD_BF16) == 0
    assert lib.ssd_linattn_bwd_workspace_bytes(_ref(d), ssd.SSD_BF16) == 0


def test_linattn_rejects_launches_past_the_grid():
    """A launch has fewer than 2^32 threads along an axis: 256 for each head of a
    sequence, three times over for the gradients."""
    d = ldims(tokens=1 << 22, nseq=1 << 20)
    assert fwd(d, cu=FAKE) == UNS and bwd(d, cu=FAKE) == UNS and step(d) == UNS
    assert lib.ssd_linattn_fwd_workspace_bytes(_ref(d), ssd.SSD_BF16) == 0
    d = ldims(tokens=1 << 22, nseq=(1 << 20) - 1)
    assert lib.ssd_linattn_fwd_workspace_bytes(_ref(d), ssd.SSD_BF16) > 0
    # (within the limits, and refused for the argument)
    assert fwd(d, cu=FAKE, ws=None) == WS and bwd(d, cu=FAKE, ws=None) == WS
    assert step(ldims(tokens=(1 << 22) - 1), q=None) == INV


def test_norms_reject_rows_past_the_grid():
    for call in (gate_fwd, gate_bwd):
        assert call(ndims(dim=1 << 28, group=1 << 14, weight_dim=1 << 28)) == UNS
        assert call(ndims(dim=1 << 27, group=1 << 14, weight_dim=1 << 27), x=None) == INV


def test_linattn_rejects_bad_arguments():
    d = ldims()
    assert fwd(None) == INV and bwd(None) == INV and step(None) == INV
    for call, names in ((fwd, ("q", "k", "v", "ld", "out")),
                        (bwd, ("q", "k", "v", "ld", "do", "dq", "dk", "dv")),
                        (step, ("q", "k", "v", "ld", "state", "out"))):
        for n in names:
            assert call(d, **{n: None}) == INV, n
            assert call(d, **{n: MISALIGNED}) == INV, n
        assert call(d, dt=2) == INV and call(d, dt=-1) == INV
    assert fwd(d, init=MISALIGNED) == INV and fwd(d, fin=MISALIGNED) == INV
    assert bwd(d, init=MISALIGNED) == INV and bwd(d, dfin=MISALIGNED) == INV
    assert bwd(d, dinit=MISALIGNED) == INV
    assert fwd(d, cu=ODD) == INV and bwd(d, cu=ODD) == INV
    # final over part of init (the whole of it is a sequence continued in place)
    assert fwd(d, init=FAKE, fin=ctypes.c_void_p(FAKE.value + 4096)) == INV
    # dinit over dfinal, whole or in part
    assert bwd(d, dfin=FAKE, dinit=FAKE) == INV
    assert bwd(d, dfin=FAKE, dinit=ctypes.c_void_p(FAKE.value + 4096)) == INV
    # sequences of equal length: tokens must divide by their number
    assert fwd(ldims(nseq=3)) == INV and bwd(ldims(nseq=3)) == INV
    assert fwd(ldims(nseq=0)) == INV and bwd(ldims(nseq=1 << 31)) == INV


@pytest.mark.parametrize("call,name", [(fwd, "ssd_linattn_fwd_workspace_bytes"),
                                       (bwd, "ssd_linattn_bwd_workspace_bytes")])
def test_linattn_rejects_small_workspace(call, name):
    for kw in ({}, dict(ngroups=4), dict(tokens=20000, nseq=1)):
        d = ldims(**kw)
        for dt in (ssd.SSD_BF16, ssd.SSD_F32):
            need = getattr(lib, name)(_ref(d), dt)
            assert need >= 16
            assert call(d, wsb=need - 1, dt=dt) == WS
            assert call(d, ws=None, dt=dt) == WS and call(d, ws=MISALIGNED, dt=dt) == WS
    assert getattr(lib, name)(None, ssd.SSD_BF16) == 0
    assert getattr(lib, name)(_ref(ldims()), 5) == 0


def add_fwd(rows=4, dim=64, eps=1e-5, **o):
    return lib.ssd_add_norm_fwd(o.get("x", FAKE), o.get("res"), o.get("s"), o.get("w"),
                                o.get("y", FAKE), o.get("ro"), rows, dim, eps,
                                o.get("xd", ssd.SSD_BF16), o.get("rd", ssd.SSD_F32), None)


def add_bwd(rows=4, dim=64, eps=1e-5, **o):
    return lib.ssd_add_norm_bwd(
        o.get("x", FAKE), o.get("res", FAKE), o.get("s"), o.get("w"), o.get("dy", FAKE),
        o.get("dro"), o.get("dx", FAKE), o.get("dres"), o.get("ds"), o.get("dw"),
        o.get("ws", FAKE), o.get("wsb", 1 << 40), rows, dim, eps, o.get("xd", ssd.SSD_BF16),
        o.get("rd", ssd.SSD_F32), None)


def test_add_norm_rejects():
    for call in (add_fwd, add_bwd):
        for kw in (dict(rows=0), dict(rows=1 << 31), dict(dim=0), dict(dim=-8), dict(eps=0.0),
                   dict(eps=-1.0), dict(eps=float("nan")), dict(xd=2), dict(rd=-1),
                   dict(x=None), dict(x=MISALIGNED), dict(res=MISALIGNED), dict(s=MISALIGNED),
                   dict(w=MISALIGNED)):
            assert call(**kw) == INV, kw
        assert call(dim=16385) == UNS
    assert add_fwd(y=None) == INV and add_fwd(ro=MISALIGNED) == INV
    for n in ("dy", "dx"):
        assert add_bwd(**{n: None}) == INV, n
    for n in ("dro", "dres", "ds", "dw"):
        assert add_bwd(**{n: MISALIGNED}) == INV, n
    assert add_bwd(ds=FAKE) == INV               # no scale, so no gradient of it
    assert add_bwd(res=None, dres=FAKE) == INV   # no residual
    need = lib.ssd_add_norm_bwd_workspace_bytes(4, 64)
    assert need > 0 and add_bwd(wsb=need - 1) == WS and add_bwd(ws=None) == WS
    assert lib.ssd_add_norm_bwd_workspace_bytes(0, 64) == 0
    assert lib.ssd_add_norm_bwd_workspace_bytes(4, 20000) == 0


def ndims(**kw):
    base = dict(rows=4, dim=128, group=64, weight_dim=64)
    base.update(kw)
    return ssd.GatedNormDims(**base)


def gate_fwd(d, eps=1e-5, **o):
    return lib.ssd_gated_norm_fwd(o.get("x", FAKE), o.get("z", FAKE), o.get("w", FAKE),
                                  o.get("y", FAKE), eps, o.get("gate", 0), 0,
                                  o.get("xd", ssd.SSD_BF16), o.get("zd", ssd.SSD_BF16),
                                  _ref(d), None)


def gate_bwd(d, eps=1e-5, **o):
    return lib.ssd_gated_norm_bwd(
        o.get("x", FAKE), o.get("z", FAKE), o.get("w", FAKE), o.get("dy", FAKE),
        o.get("dx", FAKE), o.get("dz", FAKE), o.get("dw", FAKE), o.get("ws", FAKE),
        o.get("wsb", 1 << 40), eps, o.get("gate", 0), 0, o.get("xd", ssd.SSD_BF16),
        o.get("zd", ssd.SSD_BF16), _ref(d), None)


def test_gated_norm_rejects():
    for call in (gate_fwd, gate_bwd):
        assert call(None) == INV
        for kw in (dict(rows=0), dict(dim=0), dict(group=0), dict(group=48), dict(group=256),
                   dict(weight_dim=32), dict(weight_dim=0), dict(rows=1 << 31)):
            assert call(ndims(**kw)) == INV, kw
        assert call(ndims(dim=20000, group=20000, weight_dim=20000)) == UNS
        assert call(ndims(dim=1 << 20, group=8, weight_dim=8)) == UNS
        d = ndims()
        for o in (dict(x=None), dict(x=MISALIGNED), dict(z=MISALIGNED), dict(w=MISALIGNED),
                  dict(gate=2), dict(gate=-1), dict(xd=7), dict(zd=7), dict(eps=0.0)):
            assert call(d, **o) == INV, o
    d = ndims()
    assert gate_fwd(d, y=None) == INV
    for n in ("dy", "dx"):
        assert gate_bwd(d, **{n: None}) == INV, n
    assert gate_bwd(d, z=None) == INV and gate_bwd(d, dz=None) == INV
    assert gate_bwd(d, dw=MISALIGNED) == INV
    need = lib.ssd_gated_norm_bwd_workspace_bytes(_ref(d))
    assert need > 0 and gate_bwd(d, wsb=need - 1) == WS and gate_bwd(d, ws=None) == WS
    assert lib.ssd_gated_norm_bwd_workspace_bytes(None) == 0


def test_binding_rejects_cpu_tensors_and_bad_names():
    x = torch.zeros(2, 64, 1, 64)
    with pytest.raises(ValueError):
        ssd.linattn(x, x, x, torch.zeros(1))
    with pytest.raises(ValueError):
        ssd.linattn(x[0], x[0], x[0], torch.zeros(1))
    with pytest.raises(ValueError):
        ssd.linattn_backward(x, x, x, torch.zeros(1), x)
    with pytest.raises(ValueError):
        ssd.ssd_linattn_step(x[:, 0], x[:, 0], x[:, 0], torch.zeros(1), x, x[:, 0])
    with pytest.raises(ValueError):
        ssd.add_norm(x)
    with pytest.raises(ValueError):
        ssd.gated_norm(x)
    with pytest.raises(ValueError):
        ssd._gate("relu")
