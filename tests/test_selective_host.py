"""Host-side checks of the C ABI and the binding of the operators around a selective
state space (no GPU needed).

As in test_block_host.py: every call below fails argument validation, which the
library performs on the host before any HIP call, so nothing is launched and no pointer is
touched; the module refuses to run where a GPU is visible.
"""
import ctypes
import subprocess

import pytest
import torch

if torch.cuda.is_available():
    pytest.skip("host-only validation tests use fake device pointers; "
                "not run where a GPU is visible", allow_module_level=True)

import mamba_ssd_chunked_fwd_amd as ssd  # noqa: E402
from test_kernel_scratch_host import scratch  # noqa: E402,F401

INV, UNS, WS = (ssd.SSD_ERR_INVALID_ARGUMENT, ssd.SSD_ERR_UNSUPPORTED, ssd.SSD_ERR_WORKSPACE)
lib = ssd.library()
FAKE = ctypes.c_void_p(0x7F0000000000)       # 16-byte aligned, never used
OFF4 = ctypes.c_void_p(0x7F0000000004)
OFF2 = ctypes.c_void_p(0x7F0000000002)
OFF1 = ctypes.c_void_p(0x7F0000000001)
BF16, F32 = ssd.SSD_BF16, ssd.SSD_F32


def _ref(d):
    return None if d is None else ctypes.byref(d)


def test_every_declared_function_is_exported():
    names = ssd.header_functions(ssd.SELECTIVE_HEADER_PATH)
    assert len(names) == len(set(names)) == 10
    out = subprocess.run(["nm", "-D", "--defined-only", ssd.LIB_PATH],
                         capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    for n in names:
        assert n in exported, n


def cdims(**kw):
    return ssd.ShortConvDims(**{**dict(tokens=64, nseq=2, dim=96, width=4, x_stride=0), **kw})


def conv_fwd(d, **o):
    return lib.ssd_short_conv_fwd(o.get("x", FAKE), o.get("w", FAKE), o.get("b"), o.get("init"),
                                  o.get("cu"), o.get("y", FAKE), o.get("fin"), o.get("act", 1),
                                  o.get("dt", BF16), _ref(d), None)


def conv_bwd(d, **o):
    return lib.ssd_short_conv_bwd(o.get("x", FAKE), o.get("w", FAKE), o.get("b"), o.get("init"),
                                  o.get("cu"), o.get("dy", FAKE), o.get("dfin"),
                                  o.get("dx", FAKE), o.get("dw"), o.get("db"), o.get("dinit"),
                                  o.get("ws", FAKE), o.get("wsb", 1 << 50), o.get("act", 1),
                                  o.get("dt", BF16), _ref(d), None)


def conv_step(d, **o):
    return lib.ssd_short_conv_step(o.get("x", FAKE), o.get("w", FAKE), o.get("b"),
                                   o.get("state", FAKE), o.get("y", FAKE), o.get("act", 1),
                                   o.get("dt", BF16), _ref(d), None)


CONV = (conv_fwd, conv_bwd, conv_step)


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=0), INV), (dict(tokens=1 << 31), INV), (dict(dim=0), INV), (dict(dim=-8), INV),
    (dict(width=0), INV), (dict(width=1), UNS), (dict(width=5), UNS), (dict(x_stride=95), INV),
    (dict(x_stride=-1), INV), (dict(x_stride=1 << 31), INV), (dict(dim=(1 << 20) + 1), UNS),
    (dict(tokens=1 << 30, dim=1 << 19), UNS)])
def test_conv_rejects_bad_dims(kw, expect):
    d = cdims(**kw)
    for call in CONV:
        assert call(d) == expect
    assert lib.ssd_short_conv_bwd_workspace_bytes(_ref(d)) == 0


def test_conv_rejects_bad_arguments():
    d = cdims()
    for call in CONV:
        assert call(None) == INV
        for n in ("x", "w"):
            assert call(d, **{n: None}) == INV, n
        # rows of x start on an element, everything else on 16 bytes
        assert call(d, x=OFF1) == INV and call(d, x=OFF2, dt=F32) == INV
        assert call(d, w=OFF4) == INV and call(d, b=OFF4) == INV
        assert call(d, act=2) == INV and call(d, act=-1) == INV and call(d, dt=2) == INV
    assert conv_step(d, state=None) == INV and conv_step(d, state=OFF4) == INV
    assert conv_step(d, y=None) == INV and conv_fwd(d, y=OFF4) == INV
    for n in ("init", "fin"):
        assert conv_fwd(d, **{n: OFF4}) == INV
    for n in ("init", "dfin", "dw", "db", "dinit", "dy", "dx"):
        assert conv_bwd(d, **{n: OFF4}) == INV, n
    assert conv_bwd(d, dy=None) == INV and conv_bwd(d, dx=None) == INV
    for call in (conv_fwd, conv_bwd):
        assert call(d, cu=OFF2) == INV
        assert call(cdims(nseq=3)) == INV           # 64 tokens in 3 equal sequences
        assert call(cdims(nseq=0)) == INV and call(cdims(nseq=1 << 22), cu=FAKE) == UNS
    # part of one state over the other (the whole is a sequence continued in place)
    part = ctypes.c_void_p(FAKE.value + 64)
    assert conv_fwd(d, init=FAKE, fin=part) == INV
    assert conv_bwd(d, dfin=FAKE, dinit=FAKE) == INV and conv_bwd(d, dfin=part, dinit=FAKE) == INV
    need = lib.ssd_short_conv_bwd_workspace_bytes(_ref(d))
    assert need > 0 and conv_bwd(d, wsb=need - 1) == WS
    assert conv_bwd(d, ws=None) == WS and conv_bwd(d, ws=OFF4) == WS
    assert lib.ssd_short_conv_bwd_workspace_bytes(None) == 0


def sdims(**kw):
    base = dict(tokens=64, nseq=2, dim=96, dstate=16, ngroups=2, x_stride=0, dt_stride=0,
                z_stride=0, b_stride=0, c_stride=0)
    return ssd.SelectiveScanDims(**{**base, **kw})


def _inputs(o):
    return [o.get("x", FAKE), o.get("delta", FAKE), o.get("A", FAKE), o.get("B", FAKE),
            o.get("C", FAKE), o.get("D"), o.get("z"), o.get("bias")]


def scan_fwd(d, **o):
    return lib.ssd_selective_scan_fwd(*_inputs(o), o.get("init"), o.get("cu"), o.get("y", FAKE),
                                      o.get("fin"), o.get("ws", FAKE), o.get("wsb", 1 << 60), 1,
                                      o.get("dt", BF16), _ref(d), None)


def scan_bwd(d, **o):
    return lib.ssd_selective_scan_bwd(
        *_inputs(o), o.get("init"), o.get("cu"), o.get("dy", FAKE), o.get("dfin"),
        o.get("dx", FAKE), o.get("ddt", FAKE), o.get("dA", FAKE), o.get("dB", FAKE),
        o.get("dC", FAKE), o.get("dD"), o.get("dz"), o.get("dbias"), o.get("dinit"),
        o.get("ws", FAKE), o.get("wsb", 1 << 60), 1, o.get("dt", BF16), _ref(d), None)


def scan_step(d, **o):
    return lib.ssd_selective_scan_step(*_inputs(o), o.get("state", FAKE), o.get("y", FAKE), 1,
                                       o.get("dt", BF16), _ref(d), None)


SCAN = (scan_fwd, scan_bwd, scan_step)


@pytest.mark.parametrize("kw,expect", [
    (dict(tokens=0), INV), (dict(tokens=1 << 31), INV), (dict(dim=0), INV), (dict(dstate=0), INV),
    (dict(dstate=4), UNS), (dict(dstate=24), UNS), (dict(dstate=128), UNS), (dict(ngroups=0), INV),
    (dict(ngroups=5), INV), (dict(dim=1 << 21), UNS), (dict(x_stride=95), INV),
    (dict(dt_stride=1), INV), (dict(z_stride=-96), INV), (dict(b_stride=31), INV),
    (dict(c_stride=33), INV),
    (dict(tokens=(1 << 31) - 1, dim=1 << 20, nseq=1 << 21), UNS)])
def test_scan_rejects_bad_dims(kw, expect):
    d = sdims(**kw)
    for call in SCAN:
        assert call(d) == expect
    assert lib.ssd_selective_scan_fwd_workspace_bytes(_ref(d), BF16) == 0
    assert lib.ssd_selective_scan_bwd_workspace_bytes(_ref(d), BF16) == 0


def test_scan_rejects_bad_arguments():
    d = sdims()
    for call in SCAN:
        assert call(None) == INV
        for n in ("x", "delta", "A", "B", "C"):
            assert call(d, **{n: None}) == INV, n
        for n in ("x", "delta", "z"):
            assert call(d, **{n: OFF1}) == INV and call(d, dt=F32, **{n: OFF2}) == INV, n
        for n in ("B", "C"):
            assert call(d, **{n: OFF2}) == INV, n
        for n in ("A", "D", "bias"):
            assert call(d, **{n: OFF4}) == INV, n
        assert call(d, dt=2) == INV and call(d, dt=-1) == INV
    for n in ("init", "fin", "y"):
        assert scan_fwd(d, **{n: OFF4}) == INV
    for n in ("init", "dy", "dfin", "dx", "ddt", "dA", "dB", "dC", "dD", "dbias", "dinit"):
        assert scan_bwd(d, **{n: OFF4}) == INV, n
    for n in ("dy", "dx", "ddt", "dA", "dB", "dC"):
        assert scan_bwd(d, **{n: None}) == INV, n
    assert scan_bwd(d, z=FAKE) == INV and scan_bwd(d, dz=FAKE) == INV
    assert scan_step(d, state=None) == INV and scan_step(d, state=OFF4) == INV
    assert scan_step(d, y=None) == INV and scan_fwd(d, y=None) == INV
    for call in (scan_fwd, scan_bwd):
        assert call(d, cu=OFF2) == INV and call(sdims(nseq=3)) == INV
        assert call(sdims(nseq=0)) == INV and call(sdims(nseq=1 << 22), cu=FAKE) == UNS
    part = ctypes.c_void_p(FAKE.value + 4096)
    assert scan_fwd(d, init=FAKE, fin=part) == INV
    assert scan_bwd(d, dfin=FAKE, dinit=FAKE) == INV and scan_bwd(d, dfin=part, dinit=FAKE) == INV


@pytest.mark.parametrize("kw", [{}, dict(tokens=20000, nseq=1), dict(dim=8192, nseq=64),
                                dict(dstate=64, ngroups=1)])
def test_scan_rejects_small_workspace(kw):
    d = sdims(**kw)
    for call, name in ((scan_fwd, "ssd_selective_scan_fwd_workspace_bytes"),
                       (scan_bwd, "ssd_selective_scan_bwd_workspace_bytes")):
        for dt in (BF16, F32):
            need = getattr(lib, name)(_ref(d), dt)
            assert need >= 16
            assert call(d, wsb=need - 1, dt=dt) == WS
            assert call(d, ws=None, dt=dt) == WS and call(d, ws=OFF4, dt=dt) == WS
        assert getattr(lib, name)(None, BF16) == 0 and getattr(lib, name)(_ref(d), 5) == 0


def quant(rows=4, dim=256, group=64, eps=1e-5, **o):
    return lib.ssd_add_norm_quant_fwd(
        o.get("x", FAKE), o.get("res"), o.get("s"), o.get("w"), o.get("codes", FAKE),
        o.get("scales", FAKE), o.get("ro"), rows, dim, group, eps, o.get("code", 0),
        o.get("xd", BF16), o.get("rd", F32), None)


def test_quant_rejects():
    for kw in (dict(rows=0), dict(rows=1 << 31), dict(dim=0), dict(dim=-8), dict(group=0),
               dict(group=48), dict(group=512), dict(eps=0.0), dict(eps=float("nan")),
               dict(xd=2), dict(rd=-1), dict(code=2), dict(code=-1), dict(x=None),
               dict(codes=None), dict(scales=None), dict(x=OFF4), dict(codes=OFF4),
               dict(scales=OFF4), dict(res=OFF4), dict(s=OFF4), dict(w=OFF4), dict(ro=OFF4)):
        assert quant(**kw) == INV, kw
    assert quant(dim=16385, group=16385) == UNS and quant(dim=1 << 15, group=128) == UNS
    assert quant(group=8) == UNS and quant(dim=1024, group=512) == UNS


def test_binding_rejects_cpu_tensors_and_bad_names():
    x, w = torch.zeros(1, 8, 64), torch.zeros(64, 4)
    B = torch.zeros(1, 8, 1, 16)
    A = torch.zeros(64, 16)
    with pytest.raises(ValueError, match="GPU"):
        ssd.short_conv(x, w)
    with pytest.raises(ValueError):
        ssd.short_conv(x[0], w)
    with pytest.raises(ValueError):
        ssd.short_conv_backward(x, w, None, x)
    with pytest.raises(ValueError):
        ssd.ssd_short_conv_step(x, w, None, x, x)
    with pytest.raises(ValueError, match="GPU"):
        ssd.selective_scan(x, x, A, B, B)
    with pytest.raises(ValueError):
        ssd.selective_scan(x, x, A, B[0], B)
    with pytest.raises(ValueError):
        ssd.selective_scan_backward(x, x, A[0], B, B, None, None, None, x)
    with pytest.raises(ValueError):
        ssd.ssd_selective_scan_step(x, x, A, B, B, None, None, None, A, x)
    with pytest.raises(ValueError):
        ssd.add_norm_quant(x)
    with pytest.raises(ValueError):
        ssd.add_norm_quant(x, group=48)
    with pytest.raises(ValueError):
        ssd._conv_act("relu")
    with pytest.raises(ValueError):
        ssd._quant_code(torch.uint8)


def test_row_strides():
    """Rows that are columns of a wider tensor, and layouts that have no one stride."""
    def stride(t, name="x"):
        return ssd._row_stride(name, t.shape, t.stride())

    wide = torch.zeros(2, 5, 96)
    assert stride(wide[..., 32:64]) == 96
    assert stride(wide[0, :, :32]) == 96
    assert stride(wide[:, 0, :32]) == 5 * 96      # a batch's first tokens
    assert stride(wide[:, :1, :32]) == 5 * 96
    assert stride(wide[..., 32:64].unflatten(-1, (2, 16)), "B") == 96
    assert stride(wide[0, :, 32:64].unflatten(-1, (2, 16)), "B") == 96
    for bad in (wide[:, :3], wide.transpose(1, 2), wide[..., ::2], wide[:1, :1].expand(2, 5, 96)):
        with pytest.raises(ValueError, match="pass a copy"):
            stride(bad)
    with pytest.raises(ValueError, match="pass a copy"):
        stride(wide.unflatten(-1, (2, 48))[..., :16], "B")


def conv_inputs():
    return {"x": torch.zeros(1, 8, 64), "weight": torch.zeros(64, 4), "bias": torch.zeros(64),
            "init_state": torch.zeros(1, 3, 64)}


def scan_inputs():
    x, B = torch.zeros(1, 8, 64), torch.zeros(1, 8, 1, 16)
    return {"x": x, "dt": x.clone(), "A": torch.zeros(64, 16), "B": B, "C": B.clone(),
            "D": torch.zeros(64), "z": x.clone(), "dt_bias": torch.zeros(64),
            "init_state": torch.zeros(1, 64, 16)}


def quant_inputs():
    x = torch.zeros(8, 64)
    return {"x": x, "residual": x.clone(), "res_scale": torch.zeros(64),
            "weight": torch.zeros(64)}


CALLS = [(f, n) for f, t in (("short_conv", conv_inputs), ("selective_scan", scan_inputs),
                             ("add_norm_quant", quant_inputs)) for n in t()]


@pytest.mark.parametrize("call,name", CALLS)
def test_a_lost_gradient_is_refused(call, name):
    args = {"short_conv": conv_inputs, "selective_scan": scan_inputs,
            "add_norm_quant": quant_inputs}[call]()
    args[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{call} .*{name} requires"):
        getattr(ssd, call)(**args)
    with torch.no_grad(), pytest.raises(ValueError, match="must be a GPU tensor"):
        getattr(ssd, call)(**args)


@pytest.mark.parametrize("kernel", ["scan_kernel", "scan_local_kernel", "scan_bwd_kernel",
                                    "scan_sum_bc_kernel", "scan_sum_slots_kernel",
                                    "selective_step_kernel", "short_conv_fwd_kernel",
                                    "short_conv_bwd_kernel", "short_conv_sum_kernel",
                                    "short_conv_step_kernel", "add_norm_quant_kernel"])
def test_scratch(scratch, kernel):  # noqa: F811
    sizes = {n: s for n, s in scratch.items() if kernel in n}
    assert sizes, "not in the library"
    worst = max(sizes, key=sizes.get)
    assert sizes[worst] <= 128, (worst, sizes[worst])
