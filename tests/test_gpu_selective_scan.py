"""The selective scan, its gradients and its recurrent form, against the 64-bit recurrence.

Tolerance (selective_ref.check): per token a state gets a decay (a product, an exponential
good to 2^-23, and the time step's few roundings times the exponent, of which e^-v v < 1/2
matters) and a sum; over the up to 1200 tokens that a state remembers the roundings grow
like sqrt(1200) 2^-22 < 2^-16.8.  2^-16 of the sum of absolute values."""
import pytest
import torch

import selective_ref as ref
from gpu_util import log
from selective_util import (DEV, TYPES, Guarded, Rows, dbl, dev, draw_lens, name_of, rng_of,
                            same_bits, spread)

pytestmark = pytest.mark.gpu
SUMS = 2.0 ** -16


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


def draw(i):
    rng = rng_of(900 + i)
    G = rng.choice([1, 1, 2, 3])
    c = {"i": i, "G": G, "dim": G * spread(rng, 1, 700 // G), "N": rng.choice([8, 16, 16, 32, 64]),
         "dt": rng.choice(["bf16", "fp32"]), "D": rng.random() < 0.7, "z": rng.random() < 0.7,
         "bias": rng.random() < 0.7, "softplus": rng.random() < 0.8, "init": rng.random() < 0.6,
         "dfinal": rng.random() < 0.6, "packed": rng.random() < 0.8, "wide": rng.random() < 0.5}
    return c | draw_lens(rng, spread(rng, 1, 400), c["packed"])


def named(i, **kw):
    return {**dict(i=i, G=1, dim=128, N=16, dt="fp32", D=True, z=True, bias=True, softplus=True,
                   init=True, dfinal=True, packed=True, wide=False, before=0, after=0), **kw}


NAMED = [
    named(200, dim=192, dt="bf16", lens=[1, 37, 64, 130, 0, 411], wide=True),
    named(201, dim=64, lens=[1100]),
    named(202, dim=600, G=2, lens=[33, 32, 31, 0, 1, 8, 7, 9], before=3, after=5),
    # more sequences than a search step has lanes, so many that none is cut into runs
    named(203, dim=40, N=8, lens=[2, 0, 1, 3] * 300),
    named(204, dim=1, N=64, lens=[70]),
    named(205, dim=257, N=32, dt="bf16", lens=[96, 5], wide=True),
    named(206, dim=130, G=2, N=64, lens=[64, 65], init=False, dfinal=False),
    named(207, dim=320, N=64, lens=[40]),
    # (a chain long enough to have runs of more than 32 tokens)
    named(208, dim=8256, N=8, dt="bf16", lens=[60, 20, 0, 4]),
    # (so many chains that the gradients' sequences are whole too, but for one of four times the mean)
    named(209, dim=8256, N=8, dt="bf16", lens=[40, 0, 9, 130] + [17] * 13, before=1, after=2),
    named(210, dim=4160, N=16, lens=[21] * 40, packed=False),
]


@pytest.mark.parametrize("c", NAMED + [draw(i) for i in range(32)], ids=name_of)
def test_prompts_and_gradients(ssd, c):
    log(f"[scan] {c}")
    r = Rows(c, c["i"])
    D, N, G, dt, n = c["dim"], c["N"], c["G"], TYPES[c["dt"]], len(c["lens"])
    x, xd = r(D, dtype=dt, wide=c["wide"])
    steps = dict(std=0.7, offset=0.0 if c["bias"] else -3.0) if c["softplus"] else \
        dict(std=0.02, offset=0.1)
    de, ded = r(D, dtype=dt, wide=c["wide"], **steps)
    B, Bd = r(G, N, dtype=dt, wide=c["wide"])
    C, Cd = r(G, N, dtype=dt, wide=c["wide"])
    z, zd = r(D, dtype=dt, wide=c["wide"]) if c["z"] else (None, None)
    dy, dyd = r(D, dtype=dt)
    A = -(torch.arange(1, N + 1).float() * (1 + 0.2 * r.normal(D, N)).abs())
    skip = r.normal(D) if c["D"] else None
    bias = (r.normal(D) - 3.0 if c["softplus"] else 0.01 * r.normal(D)) if c["bias"] else None
    init = r.normal(n, D, N) if c["init"] else None
    dfinal = r.normal(n, D, N) if c["dfinal"] else None
    args = (xd, ded, A.double(), Bd, Cd, dbl(skip), zd, dbl(bias), c["lens"], c["softplus"],
            dbl(init), dyd, dbl(dfinal))
    want, size = ref.scan(*args), ref.scan(*args, size=True)
    ins = (x, de, dev(A), B, C, dev(skip), z, dev(bias))
    out, results = Guarded(), []
    f32 = torch.float32
    for rep in range(2):
        y, dx, ddt = (out(x.shape, dt) for _ in range(3))
        dz = out(x.shape, dt) if c["z"] else None
        dB, dC = (out(B.shape, dt) for _ in range(2))
        final, dinit = (out((n, D, N), f32) for _ in range(2))
        dA, dD, db = out((D, N), f32), out((D,), f32), out((D,), f32)
        d = ssd._scan_prompt_args(*ins, None, r.cu)[0]
        ws = [out((ssd.selective_scan_workspace_bytes(d, dt, back),), torch.uint8)
              for back in (False, True)]
        start = dev(init)
        if rep and init is not None:      # the second time in place
            final.copy_(start)
            start = final
        ssd.ssd_selective_scan_fwd(*ins, start, r.cu, y, final, ws[0], c["softplus"])
        ssd.ssd_selective_scan_bwd(*ins, dev(init), r.cu, dy, dev(dfinal), dx, ddt, dA, dB, dC,
                                   dD, dz, db, dinit, ws[1], c["softplus"])
        results.append({"y": y, "final": final, "dx": dx, "ddt": ddt, "dA": dA, "dB": dB,
                        "dC": dC, "dD": dD, "dz": dz, "ddt_bias": db, "dinit": dinit})
        if dz is None:
            del results[-1]["dz"]
    out.check()
    for m, t in results[0].items():
        assert same_bits(t, results[1][m]), m
    got = {m: r.cut(m, t) if m in ("y", "dx", "ddt", "dB", "dC", "dz") else t
           for m, t in results[0].items()}
    worst = ref.check(got, want, size, SUMS)
    log("  of the tolerance " + ", ".join(f"{m} {v:.2f}" for m, v in worst.items()))


@pytest.mark.parametrize("b,D,N,G,dt", [
    (1, 2560, 16, 1, "bf16"), (7, 33, 8, 3, "bf16"), (200, 136, 16, 1, "fp32"),
    (3, 1, 64, 1, "fp32"), (65, 48, 32, 2, "bf16")])
@pytest.mark.parametrize("full", [True, False])
def test_step(ssd, b, D, N, G, dt, full):
    g = torch.Generator().manual_seed(b + D)
    dt = TYPES[dt]

    def rows(*shape, std=1.0):
        t = (torch.randn(b, *shape, generator=g) * std).to(dt).to(DEV)
        if not full:
            return t
        wide = torch.full((b, t[0].numel() + 10), float("nan"), dtype=dt, device=DEV)
        wide[:, 4:4 + t[0].numel()] = t.flatten(1)
        return wide[:, 4:4 + t[0].numel()].unflatten(-1, shape)

    x, de, B, C = rows(D), rows(D, std=0.7), rows(G, N), rows(G, N)
    z = rows(D) if full else None
    A = -torch.rand(D, N, generator=g) * N
    skip, bias = (torch.randn(D, generator=g) - 2 if full else None for _ in range(2))
    state = torch.randn(b, D, N, generator=g)
    args = (dbl(x), dbl(de), A.double(), dbl(B), dbl(C), dbl(skip), dbl(z), dbl(bias), [1] * b,
            True, state.double())
    want, size = ref.scan(*args), ref.scan(*args, size=True)
    out = Guarded()
    y, s = out((b, D), dt), out((b, D, N), torch.float32)
    s.copy_(state)
    ssd.ssd_selective_scan_step(x, de, dev(A), B, C, dev(skip), z, dev(bias), s, y)
    out.check()
    ref.check({"y": y, "final": s}, want, size, 2.0 ** -20)


def block_inputs(T, D=96, N=16, seed=0, n=1, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)

    def rows(*shape, std=1.0):
        return (torch.randn(n, T, *shape, generator=g) * std).to(dtype).to(DEV)

    return [rows(D), rows(D, std=0.5), -torch.rand(D, N, generator=g).to(DEV) * N, rows(1, N),
            rows(1, N), torch.randn(D, generator=g).to(DEV), rows(D),
            (torch.randn(D, generator=g) - 3).to(DEV)]


def test_steps_continue_a_prompt(ssd):
    a = block_inputs(90, n=2)
    whole, last = ssd.selective_scan(*a)
    head = [t[:, :77].contiguous() if t.dim() > 2 else t for t in a]
    y, state = ssd.selective_scan(*head)
    for t in range(77, 90):
        out = torch.empty(2, 96, device=DEV)
        ssd.ssd_selective_scan_step(*(v[:, t] if v.dim() > 2 else v for v in a), state, out)
        assert float((out - whole[:, t]).norm() / whole[:, t].norm()) < 1e-5
    assert float((state - last).norm() / last.norm()) < 1e-5


def test_gradients_against_differences(ssd):
    """The forward call's own differences along one direction of each input."""
    a = block_inputs(70, D=64)
    g = torch.Generator().manual_seed(5)
    init = torch.randn(1, 64, 16, generator=g).to(DEV)
    dy, dfinal = torch.randn(1, 70, 64, generator=g).to(DEV), torch.randn(1, 64, 16,
                                                                         generator=g).to(DEV)
    grads = ssd.selective_scan_backward(*a, dy, dfinal, init)
    every = a + [init]

    def value(ins):
        y, final = ssd.selective_scan(*ins[:8], ins[8])
        return float((y.double() * dy).sum() + (final.double() * dfinal).sum())

    for i, (t, grad) in enumerate(zip(every, grads)):
        # along the gradient's signs the slope is the sum of its absolute values; the values'
        # own rounding, some 1e-6 of sums of sqrt(5000) terms, is well below 1% of it
        step = grad.sign() * 1e-2 * (t.abs() + 0.01 if i == 2 else 1.0)
        ins = list(every)
        ins[i] = t + step
        up = value(ins)
        ins[i] = t - step
        slope = (up - value(ins)) / 2
        want = float((grad.double() * step).sum())
        log(f"  {i}: {slope:.6g} against {want:.6g}")
        assert abs(slope - want) <= 0.02 * abs(want), i


def test_values_that_are_not_finite_stay_in_their_sequence(ssd):
    """... and reach no token before them."""
    a = block_inputs(120)
    cu = torch.tensor([0, 40, 80, 120], dtype=torch.int32, device=DEV)
    clean, _ = ssd.selective_scan(*a, None, cu)
    for i in (0, 1, 3, 4):
        b = list(a)
        b[i] = a[i].clone()
        b[i][0, 60] = float("inf") if i == 0 else float("nan")
        y, final = ssd.selective_scan(*b, None, cu)
        assert same_bits(y[0, :60], clean[0, :60]) and same_bits(y[0, 80:], clean[0, 80:]), i
        assert torch.isfinite(final[0]).all() and torch.isfinite(final[2]).all(), i
        assert not torch.isfinite(y[0, 60]).any(), i
        grads = ssd.selective_scan_backward(*b, torch.ones_like(a[0]), None, None, cu)
        for t in (grads[0], grads[1], grads[3], grads[4], grads[6]):
            assert torch.isfinite(t[0, :40]).all() and torch.isfinite(t[0, 80:]).all(), i


def test_decays_from_none_to_no_memory(ssd):
    a = block_inputs(200, dtype=torch.float32)
    a[2] = a[2].clone()
    a[2][:, 0] = 0.0                   # never forgets
    a[2][:, 1] = -1e30                 # keeps nothing
    a[2][:, 2] = -3e4                  # denormal powers
    want = ref.scan(*(dbl(t)[0] if t.dim() > 2 else dbl(t) for t in a), [200])
    y, final = ssd.selective_scan(*a)
    assert torch.isfinite(y).all() and torch.isfinite(final).all()
    assert float((y[0].double().cpu() - want["y"]).norm() / want["y"].norm()) < 1e-5
    grads = ssd.selective_scan_backward(*a, torch.ones_like(y))
    assert all(torch.isfinite(t).all() for t in grads if t is not None)


def test_decays_next_to_the_largest_finite_number(ssd):
    """A times log2(e) is not finite, and tokens past a run's end have no time: their decay is
    still 1."""
    a = block_inputs(13, dtype=torch.float32)
    a[2] = a[2].clone()
    a[2][:, 0], a[2][:, 1] = -3.2e38, -3.4e38
    dy = torch.randn(a[0].shape, generator=torch.Generator().manual_seed(4)).to(DEV)
    args = [dbl(t)[0] if t.dim() > 2 else dbl(t) for t in a]
    want = ref.scan(*args, [13], True, None, dbl(dy)[0])
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")
    grads = dict(zip(names, ssd.selective_scan_backward(*a, dy)))
    y, _ = ssd.selective_scan(*a)
    for m, t in [("y", y), *grads.items()]:
        got = t.double().cpu().reshape(want[m].shape)
        assert float((got - want[m]).norm()) <= 1e-5 * float(want[m].norm()), m


def test_entries_outside_the_tokens_are_the_nearer_end(ssd):
    a = block_inputs(100)
    cu = torch.tensor([0, 11, 100], dtype=torch.int32, device=DEV)
    off = torch.tensor([-5, 11, 1 << 30], dtype=torch.int32, device=DEV)
    for s, t in zip(ssd.selective_scan(*a, None, cu), ssd.selective_scan(*a, None, off)):
        assert same_bits(s, t)


def test_rows_more_than_2_31_elements_apart(ssd):
    """Inputs that are columns of a tensor of more than 2^31 elements."""
    T, wide = 2100, 1 << 20
    a = block_inputs(T, D=64, dtype=torch.bfloat16)
    big = torch.zeros(1, T, wide, dtype=torch.bfloat16, device=DEV)
    b, at = list(a), wide
    for i in (0, 1, 3, 4, 6):
        n = a[i][0, 0].numel()
        at -= n
        big[..., at:at + n] = a[i].flatten(2)
        b[i] = big[..., at:at + n] if a[i].dim() == 3 else \
            big[..., at:at + n].unflatten(-1, a[i].shape[2:])
    for s, t in zip(ssd.selective_scan(*a), ssd.selective_scan(*b)):
        assert same_bits(s, t)
    dy = torch.randn_like(a[0])
    for s, t in zip(ssd.selective_scan_backward(*a, dy), ssd.selective_scan_backward(*b, dy)):
        assert (s is None and t is None) or same_bits(s, t)


def test_more_than_2_31_elements(ssd):
    """Two sequences, the second behind more than 2^31 elements of every row-shaped tensor:
    what it gives alone, but for roundings (the calls cut it into other runs)."""
    D, last, dt = 5120, 300, torch.bfloat16
    T = (1 << 31) // D + 2 * last
    g = torch.Generator(device=DEV).manual_seed(8)

    def rows(*shape):
        return torch.randn(1, T, *shape, generator=g, device=DEV, dtype=dt)

    x, de, z, dy, B, C = rows(D), rows(D), rows(D), rows(D), rows(1, 8), rows(1, 8)
    A = -torch.arange(1, 9, device=DEV).float().repeat(D, 1)
    bias = torch.full((D,), -3.0, device=DEV)
    ins = (x, de, A, B, C, bias, z, bias)
    cu = torch.tensor([0, T - last, T], dtype=torch.int32, device=DEV)
    tail = [t[:, -last:] if t.dim() > 2 else t for t in ins]
    y, final = ssd.selective_scan(*ins, None, cu)
    want, state = ssd.selective_scan(*tail)
    assert _near(y[:, -last:], want) < 2 ** -8 and _near(final[1:], state) < 2 ** -16
    del y
    grads = ssd.selective_scan_backward(*ins, dy, None, None, cu)
    wants = ssd.selective_scan_backward(*tail, dy[:, -last:].contiguous())
    for i in (0, 1, 3, 4, 6):
        assert _near(grads[i][:, -last:], wants[i]) < 2 ** -8, i
        assert torch.isfinite(grads[i][:, :8]).all()


def _near(got, want):
    got, want = got.double(), want.double()
    return float((got - want).norm() / want.norm())


def test_parameters_are_tensors_too(ssd):
    a = block_inputs(20)
    b = [torch.nn.Parameter(t) if t.dim() < 3 else t for t in a]
    with torch.no_grad():
        for s, t in zip(ssd.selective_scan(*a), ssd.selective_scan(*b)):
            assert same_bits(s, t)
    with pytest.raises(ValueError, match="A requires a gradient"):
        ssd.selective_scan(*b)
