"""The short causal convolution of packed sequences, its gradients and its form for single
tokens, against the 64-bit formulas.

Tolerance (selective_ref.check): a value is a sum of at most five terms, with a gate whose
exponential and reciprocal are good to 2^-22: 2^-20 of the sum of absolute values; the
parameters' gradients are sums over up to 2000 tokens, whose roundings grow like
sqrt(2000) 2^-24 < 2^-18.  2^-18 for all.  States of x's own values are equal."""
import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_util import (DEV, TYPES, Guarded, Rows, dbl, dev, draw_lens, name_of, rng_of,
                            same_bits, spread)

pytestmark = pytest.mark.gpu
SUMS = 2.0 ** -18


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


def draw(i):
    rng = rng_of(500 + i)
    c = {"i": i, "dim": spread(rng, 1, 2100), "W": rng.choice([2, 3, 4]),
         "dt": rng.choice(["bf16", "fp32"]), "act": rng.choice(["silu", None]),
         "bias": rng.random() < 0.7, "init": rng.random() < 0.6, "dfinal": rng.random() < 0.6,
         "packed": rng.random() < 0.8, "wide": rng.random() < 0.5}
    if rng.random() < 0.6:
        c["dim"] = max(8, c["dim"] // 8 * 8)
    return c | draw_lens(rng, spread(rng, 1, 600), c["packed"])


NAMED = [
    {"i": 100, "dim": 1536, "W": 4, "dt": "bf16", "act": "silu", "bias": True, "init": True,
     "dfinal": True, "packed": True, "wide": True, "lens": [1, 37, 64, 130, 0, 411],
     "before": 0, "after": 0},
    {"i": 101, "dim": 72, "W": 4, "dt": "fp32", "act": "silu", "bias": True, "init": True,
     "dfinal": True, "packed": True, "wide": False, "lens": [0, 1, 2, 3, 4, 5, 0], "before": 2,
     "after": 9},
    {"i": 102, "dim": 8, "W": 4, "dt": "bf16", "act": None, "bias": False, "init": False,
     "dfinal": True, "packed": True, "wide": False, "lens": [2000], "before": 0, "after": 0},
    {"i": 103, "dim": 16, "W": 3, "dt": "fp32", "act": "silu", "bias": True, "init": True,
     "dfinal": False, "packed": True, "wide": False, "lens": [2, 0, 1] * 120, "before": 0,
     "after": 1},
]


@pytest.mark.parametrize("c", NAMED + [draw(i) for i in range(28)], ids=name_of)
def test_prompts_and_gradients(ssd, c):
    log(f"[conv] {c}")
    r = Rows(c, c["i"])
    D, W, dt, n = c["dim"], c["W"], TYPES[c["dt"]], len(c["lens"])
    x, xd = r(D, dtype=dt, wide=c["wide"])
    dy, dyd = r(D, dtype=dt)
    w, b = r.normal(D, W), r.normal(D) if c["bias"] else None
    init = r.normal(n, W - 1, D, dtype=dt) if c["init"] else None
    dfinal = r.normal(n, W - 1, D, dtype=dt) if c["dfinal"] else None
    args = (xd, w.double(), dbl(b), c["lens"], c["act"] == "silu", dbl(init), dyd, dbl(dfinal))
    want, size = ref.conv(*args), ref.conv(*args, size=True)
    out, results = Guarded(), []
    for rep in range(2):
        y, dx = out(x.shape, dt), out(x.shape, dt)
        final, dinit = out((n, W - 1, D), dt), out((n, W - 1, D), dt)
        dw, db = out((D, W), torch.float32), out((D,), torch.float32)
        d = ssd._conv_args(x, dev(w), dev(b), None, r.cu)[0]
        ws = out((ssd.short_conv_workspace_bytes(d),), torch.uint8)
        start = dev(init)
        if rep and init is not None:      # the second time in place
            final.copy_(start)
            start = final
        ssd.ssd_short_conv_fwd(x, dev(w), dev(b), start, r.cu, y, final, c["act"])
        ssd.ssd_short_conv_bwd(x, dev(w), dev(b), dev(init), r.cu, dy, dev(dfinal), dx, dw, db,
                               dinit, ws, c["act"])
        results.append({"y": y, "final": final, "dx": dx, "dweight": dw, "dbias": db,
                        "dinit": dinit})
    out.check()
    for m, t in results[0].items():
        assert same_bits(t, results[1][m]), m
    got = {m: r.cut(m, t) if m in ("y", "dx") else t for m, t in results[0].items()}
    worst = ref.check(got, want, size, SUMS, own=("final",))
    log("  of the tolerance " + ", ".join(f"{m} {v:.2f}" for m, v in worst.items()))


@pytest.mark.parametrize("b,D,W,dt,act", [
    (1, 2560, 4, "bf16", "silu"), (7, 33, 4, "bf16", "silu"), (200, 136, 3, "fp32", None),
    (3, 1, 2, "fp32", "silu"), (65, 1048, 2, "bf16", None)])
@pytest.mark.parametrize("wide", [True, False])
def test_step(ssd, b, D, W, dt, act, wide):
    g = torch.Generator().manual_seed(b + D)
    dt = TYPES[dt]
    x = torch.randn(b, 2 * D if wide else D, generator=g).to(dt).to(DEV)[:, -D:]
    w, bias = torch.randn(D, W, generator=g), torch.randn(D, generator=g)
    state = torch.randn(b, W - 1, D, generator=g).to(dt)
    args = (dbl(x), w.double(), bias.double(), [1] * b, act == "silu", state.double())
    want, size = ref.conv(*args), ref.conv(*args, size=True)
    out = Guarded()
    y, s = out((b, D), dt), out((b, W - 1, D), dt)
    s.copy_(state)
    ssd.ssd_short_conv_step(x, dev(w), dev(bias), s, y, act)
    out.check()
    ref.check({"y": y, "final": s}, want, size, SUMS, own=("final",))


def test_steps_continue_a_prompt(ssd):
    """Token by token from a prompt's final state gives what the whole prompt gives."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 40, 64, generator=g).to(DEV)
    w, b = torch.randn(64, 4, generator=g).to(DEV), torch.randn(64, generator=g).to(DEV)
    whole, last = ssd.short_conv(x, w, b)
    y, state = ssd.short_conv(x[:, :31].contiguous(), w, b)
    assert same_bits(y, whole[:, :31])
    for t in range(31, 40):
        out = torch.empty(2, 64, device=DEV)
        ssd.ssd_short_conv_step(x[:, t], w, b, state, out)
        assert same_bits(out, whole[:, t])
    assert same_bits(state, last)


def test_values_that_are_not_finite_stay_in_their_sequence(ssd):
    """... and reach no token before them."""
    x = torch.randn(1, 30, 24, device=DEV)
    w = torch.randn(24, 4, device=DEV)
    cu = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device=DEV)
    clean, _ = ssd.short_conv(x, w, cu_seqlens=cu)
    x[0, 14] = float("nan")
    y, final = ssd.short_conv(x, w, cu_seqlens=cu)
    assert same_bits(y[0, :14], clean[0, :14]) and same_bits(y[0, 18:], clean[0, 18:])
    assert torch.isnan(y[0, 14:18]).all() and torch.isfinite(final).all()
    dy = torch.randn_like(x)
    dx = ssd.short_conv_backward(x, w, None, dy, cu_seqlens=cu)[0]
    assert torch.isfinite(dx[0, :10]).all() and torch.isfinite(dx[0, 20:]).all()


def test_entries_outside_the_tokens_are_the_nearer_end(ssd):
    x, w = torch.randn(1, 30, 16, device=DEV), torch.randn(16, 3, device=DEV)
    cu = torch.tensor([0, 11, 30], dtype=torch.int32, device=DEV)
    off = torch.tensor([-5, 11, 1 << 30], dtype=torch.int32, device=DEV)
    for a, b in zip(ssd.short_conv(x, w, cu_seqlens=cu), ssd.short_conv(x, w, cu_seqlens=off)):
        assert same_bits(a, b)


def test_more_than_2_31_elements(ssd):
    """Rows far out, of tensors with more than 2^31 elements."""
    D, T = 2056, (1 << 20) + 77
    w, b = torch.randn(D, 4, device=DEV), torch.randn(D, device=DEV)
    x = torch.zeros(1, T, D, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(1, 100, D, device=DEV).to(torch.bfloat16)
    x[:, -100:] = tail
    cu = torch.tensor([0, T - 100, T], dtype=torch.int32, device=DEV)
    y, final = ssd.short_conv(x, w, b, cu_seqlens=cu)
    want, last = ssd.short_conv(tail, w, b)
    assert same_bits(y[:, -100:], want) and same_bits(final[1:], last)
    assert (y[0, :-100] == y[0, 0]).all()
    dx = ssd.short_conv_backward(x, w, b, y, cu_seqlens=cu)[0]
    want = ssd.short_conv_backward(tail, w, b, y[:, -100:])[0]
    assert same_bits(dx[:, -100:], want)
