"""The residual add and norm with its output in 8 bits, against the 64-bit formula: codes
are equal (everything before them is formed in 64 bits; a value within 1e-10 of a border,
where two 64-bit orders of summation may differ, may take either neighbour), scales are
good to one rounding (2^-24), the stream to one rounding of its type."""
import math
from fractions import Fraction

import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_util import DEV, TYPES, Guarded, dbl, name_of, rng_of, spread

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -17
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


def draw(i):
    rng = rng_of(300 + i)
    group = rng.choice([0, 0, 16, 32, 64, 128, 256])
    dim = spread(rng, 1, 16384)
    if group:
        dim = max(1, dim // group) * group
    return {"i": i, "rows": spread(rng, 1, 200), "dim": dim, "group": group or dim,
            "code": rng.choice(["e4m3", "int8"]), "xt": rng.choice(["bf16", "fp32"]),
            "rt": rng.choice(["bf16", "fp32"]), "residual": rng.random() < 0.8,
            "scale": rng.random() < 0.5, "weight": rng.random() < 0.8,
            "in_place": rng.random() < 0.5}


NAMED = [dict(i=90, rows=3, dim=2560, group=2560, code="e4m3", xt="bf16", rt="bf16",
              residual=True, scale=False, weight=True, in_place=False),
         dict(i=91, rows=5000, dim=128, group=128, code="int8", xt="bf16", rt="fp32",
              residual=True, scale=True, weight=True, in_place=True),
         dict(i=92, rows=17, dim=16384, group=256, code="e4m3", xt="fp32", rt="fp32",
              residual=True, scale=True, weight=True, in_place=False),
         dict(i=93, rows=9, dim=16383, group=16383, code="e4m3", xt="bf16", rt="fp32",
              residual=True, scale=True, weight=True, in_place=False)]


@pytest.mark.parametrize("c", NAMED + [draw(i) for i in range(36)], ids=name_of)
def test_codes(ssd, c):
    log(f"[quant] {c}")
    g = torch.Generator().manual_seed(c["i"])
    rows, D, group, kind = c["rows"], c["dim"], c["group"], CODES[c["code"]]
    dt, rdt = TYPES[c["xt"]], TYPES[c["rt"]]

    def normal(*shape, dtype=torch.float32, there=True):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV) if there else None

    x, res = normal(rows, D, dtype=dt), normal(rows, D, dtype=rdt, there=c["residual"])
    s, w = normal(D, there=c["scale"]), normal(D, there=c["weight"])
    want = ref.quant(dbl(x), dbl(res), dbl(s), dbl(w), EPS, group, kind)
    out = Guarded()
    codes, scales = out((rows, D), kind), out((rows, D // group), torch.float32)
    h = out((rows, D), rdt if c["residual"] else dt)
    if c["in_place"] and res is not None:
        h.copy_(res)
        res = h
    ssd.ssd_add_norm_quant_fwd(x, res, s, w, codes, scales, h, EPS)
    out.check()
    got = dbl(codes)
    off = (got != want["codes"]).nonzero()
    for i in off.tolist():
        v = want["v"][tuple(i)]
        middle = (got[tuple(i)] + want["codes"][tuple(i)]) / 2
        assert abs(v - middle) <= 1e-10 * abs(middle), (i, float(v), float(got[tuple(i)]))
    assert len(off) <= 2
    err = (dbl(scales) - want["scales"]).abs()
    assert (err <= 2.0 ** -24 * 1.001 * want["scales"] + 2.0 ** -149).all()
    half = 2.0 ** -8 if h.dtype == torch.bfloat16 else 2.0 ** -24
    assert ((dbl(h) - want["h"]).abs() <= half * 1.001 * want["h"].abs() + 2.0 ** -149).all()


def test_rows_of_zeros_and_values_that_are_not_finite(ssd):
    x = torch.randn(6, 256, device=DEV)
    x[1] = 0.0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    for kind in CODES.values():
        codes, scales, h = ssd.add_norm_quant(x, dtype=kind, group=64)
        y = codes.float().view(6, 4, 64) * scales[..., None]
        plain, _ = ssd.add_norm(x)
        assert (codes[1].float() == 0).all() and (scales[1] == 0).all()
        assert not torch.isfinite(scales[2]).any()                  # the whole row
        assert not torch.isfinite(scales[3, 3]) and not torch.isfinite(y[3, 3]).any()
        for r in (0, 4, 5):
            err = (y[r].flatten() - plain[r]).abs()
            step = scales[r].repeat_interleave(64) / 2 * (1.001 if kind == torch.int8 else 32.04)
            assert (err <= step).all(), r
        # the other groups of a row with an infinity are zeros, as add_norm gives
        assert (y[3, :3] == plain[3].view(4, 64)[:3]).all()


def test_leading_dimensions_and_wrong_arguments(ssd):
    x = torch.randn(2, 3, 64, device=DEV).to(torch.bfloat16)
    codes, scales, h = ssd.add_norm_quant(x)
    assert codes.shape == x.shape and scales.shape == (2, 3, 1) and h.shape == x.shape
    with pytest.raises(ValueError):
        ssd.add_norm_quant(x, dtype=torch.uint8)
    with pytest.raises(ssd.SsdError):
        ssd.add_norm_quant(x, group=8)
    with pytest.raises(ValueError):
        ssd.ssd_add_norm_quant_fwd(x, None, None, None, codes, scales[0], None)


@pytest.mark.parametrize("code,top", [("e4m3", 448), ("int8", 127)])
@pytest.mark.parametrize("group", [16, 80])
def test_values_on_a_border_go_to_the_even_code(ssd, code, top, group):
    """Rows of small whole numbers, whose quotients by the largest lie on borders again and
    again: what exact fractions give."""
    g = torch.Generator().manual_seed(group)
    x = torch.randint(-24, 25, (300, 80), generator=g)
    codes, scales, _ = ssd.add_norm_quant(x.to(torch.bfloat16).to(DEV), dtype=CODES[code],
                                          group=group)
    got, ties = dbl(codes).tolist(), 0
    for row, values in enumerate(x.tolist()):
        for at in range(0, 80, group):
            most = max(abs(v) for v in values[at:at + group])
            for i in range(at, at + group):
                v = Fraction(top * values[i], most)
                unit = Fraction(1)
                if code == "e4m3" and v:
                    unit = Fraction(2) ** (math.floor(math.log2(abs(v))) - 3)
                ties += (v / unit) % 1 == Fraction(1, 2)
                assert got[row][i] == float(round(v / unit) * unit), (row, i, v)
    assert ties > 100
