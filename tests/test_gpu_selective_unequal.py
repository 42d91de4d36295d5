"""The selective scan and its gradients over packs of one long sequence and many short ones, of
which the short are walked whole and the long one is cut, against the 64-bit recurrence.

Groups of one or two channels make many chains of few channels.  Tolerance as in
test_gpu_selective_scan.py: 2^-16 of the sum of absolute values, plus each output's rounding."""
import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_util import Guarded, Rows, TYPES, dbl, dev, name_of, same_bits

pytestmark = pytest.mark.gpu
SUMS = 2.0 ** -16


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


CASES = [
    # forward 1152 chains: up to 148 tokens whole, the others in runs of 24
    dict(i=1, dim=128, G=128, N=8, dt="fp32", lens=[1000, 0, 150, 1, 60, 7, 0, 33, 200],
         before=0, after=0),
    # the same in pairs of channels, behind rows of no sequence that would have slots of their own
    dict(i=2, dim=256, G=128, N=16, dt="bf16", lens=[148, 30, 800, 1, 0, 9, 149, 24, 25],
         before=77, after=5),
    # gradients too (2816 chains): up to 300 tokens whole, the others in runs of 144
    dict(i=3, dim=256, G=256, N=8, dt="fp32",
         lens=[290, 0, 150, 2000, 8, 1, 100, 300, 144, 7, 0], before=0, after=0),
    # more sequences than a search step has lanes
    dict(i=4, dim=512, G=8, N=16, dt="bf16", lens=[3] * 100 + [700] + [0, 5] * 50, before=1,
         after=60),
    # all tokens in the last of many
    dict(i=5, dim=192, G=96, N=8, dt="fp32", lens=[0] * 40 + [500], before=0, after=0),
]


@pytest.mark.parametrize("c", CASES, ids=name_of)
def test_one_long_sequence_among_many(ssd, c):
    log(f"[unequal] {c}")
    c = c | {"packed": True}
    r = Rows(c, c["i"])
    D, N, G, dt, n = c["dim"], c["N"], c["G"], TYPES[c["dt"]], len(c["lens"])
    x, xd = r(D, dtype=dt)
    de, ded = r(D, dtype=dt, std=0.7)
    B, Bd = r(G, N, dtype=dt)
    C, Cd = r(G, N, dtype=dt)
    z, zd = r(D, dtype=dt)
    dy, dyd = r(D, dtype=dt)
    A = -(torch.arange(1, N + 1).float() * (1 + 0.2 * r.normal(D, N)).abs())
    skip, bias = r.normal(D), r.normal(D) - 3.0
    init, dfinal = r.normal(n, D, N), r.normal(n, D, N)
    args = (xd, ded, A.double(), Bd, Cd, dbl(skip), zd, dbl(bias), c["lens"], True, dbl(init), dyd,
            dbl(dfinal))
    want, size = ref.scan(*args), ref.scan(*args, size=True)
    ins = (x, de, dev(A), B, C, dev(skip), z, dev(bias))
    out, results = Guarded(), []
    f32 = torch.float32
    d = ssd._scan_prompt_args(*ins, None, r.cu)[0]
    for rep in range(2):
        got = {m: out(x.shape, dt) for m in ("y", "dx", "ddt", "dz")}
        got |= {m: out(B.shape, dt) for m in ("dB", "dC")}
        got |= {m: out((n, D, N), f32) for m in ("final", "dinit")}
        got |= {"dA": out((D, N), f32), "dD": out((D,), f32), "ddt_bias": out((D,), f32)}
        ws = [out((ssd.selective_scan_workspace_bytes(d, dt, back),), torch.uint8)
              for back in (False, True)]
        start = dev(init)
        if rep:                            # the second time in place
            got["final"].copy_(start)
            start = got["final"]
        ssd.ssd_selective_scan_fwd(*ins, start, r.cu, got["y"], got["final"], ws[0])
        ssd.ssd_selective_scan_bwd(*ins, dev(init), r.cu, dy, dev(dfinal), got["dx"], got["ddt"],
                                   got["dA"], got["dB"], got["dC"], got["dD"], got["dz"],
                                   got["ddt_bias"], got["dinit"], ws[1])
        results.append(got)
    out.check()
    for m, t in results[0].items():
        assert same_bits(t, results[1][m]), m
    rows = ("y", "dx", "ddt", "dB", "dC", "dz")
    got = {m: r.cut(m, t) if m in rows else t for m, t in results[0].items()}
    worst = ref.check(got, want, size, SUMS)
    log("  of the tolerance " + ", ".join(f"{m} {v:.2f}" for m, v in worst.items()))
