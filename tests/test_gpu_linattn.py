"""Linear attention with a decay for each head (ssd_linattn_fwd, _bwd, _step)
against the token-by-token recurrence and its adjoint in 64 bits.

Tolerances, on the 2-norm of the difference over that of the result, with
h = 2^-8 the largest relative error of a rounding to bf16 (its root mean
square over random values is below h / sqrt(3)) and e = 2^-24 that of fp32:
* bf16 outputs: each is a sum of products of which two operands may have been
  rounded to bf16 (the masked scores and the state), and is rounded once
  itself.  The three roundings are independent, so the 2-norm is at most
  sqrt(3) h / sqrt(3) = h.
* fp32 states from bf16 inputs: the decayed operand is split into two bf16
  terms, which leaves at most 2^-17 of each product (h of a remainder of h,
  halved), and a few hundred fp32 sums: 2^-17.
* everything from fp32 inputs: products and sums in fp32 over up to n terms,
  whose roundings grow like sqrt(n) e at most; n <= 1200 here and the decays
  add a few: 64 e.
"""
import numpy as np
import pytest
import torch

import block_ref
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H8 = 2.0 ** -8
TOL = {torch.bfloat16: H8, torch.float32: 64 * 2.0 ** -24}
STATE_TOL = {torch.bfloat16: 2.0 ** -17, torch.float32: 64 * 2.0 ** -24}
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


def make(lens, H, G, K, V, dtype, seed, init=True, decays=None, before=0, after=0):
    """Inputs of a packed call on the CPU; `before` and `after` rows of NaN
    around the sequences belong to none of them."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    dt = DTYPES[dtype]

    def rows(n, d):
        x = torch.randn(T + before + after, n, d, generator=g)
        x[:before] = float("nan")
        x[T + before:] = float("nan")
        return x.to(dt)

    s = {"q": rows(G, K), "k": rows(G, K), "v": rows(H, V), "do": rows(H, V)}
    s["ld"] = (-torch.exp2(-8.0 * torch.arange(1, H + 1) / H) if decays is None
               else torch.tensor(decays, dtype=torch.float32))
    n = len(lens)
    s["init"] = torch.randn(n, H, K, V, generator=g) if init else None
    s["dfinal"] = torch.randn(n, H, K, V, generator=g) if init else None
    s["cu"] = torch.tensor(np.cumsum([before] + list(lens)), dtype=torch.int32)
    s |= {"lens": list(lens), "scale": K ** -0.5, "before": before, "T": T}
    return s


def reference(s, backward=True):
    cut = slice(s["before"], s["before"] + s["T"])
    q, k, v, do = (s[n][cut].double() for n in ("q", "k", "v", "do"))
    return block_ref.linattn(q, k, v, s["ld"], s["lens"], s["scale"], s["init"],
                             do if backward else None, s["dfinal"])


def on_gpu(s):
    return {n: (x.to(DEV) if isinstance(x, torch.Tensor) else x) for n, x in s.items()}


def forward(ssd, d):
    o, final = ssd.linattn(d["q"][None], d["k"][None], d["v"][None], d["ld"], d["init"], d["cu"],
                           d["scale"])
    return {"o": o[0], "final": final}


def backward(ssd, d):
    dq, dk, dv, dinit = ssd.linattn_backward(
        d["q"][None], d["k"][None], d["v"][None], d["ld"], d["do"][None], d["dfinal"], d["init"],
        d["cu"], d["scale"])
    return {"dq": dq[0], "dk": dk[0], "dv": dv[0], "dinit": dinit}


def check(got, ref, dtype, cut=slice(None)):
    for n, g in got.items():
        states = n in ("final", "dinit")
        g = g.double().cpu() if states else g[cut].double().cpu()
        r = ref[n]
        assert g.shape == r.shape, n
        assert torch.isfinite(g).all(), n
        if r.numel() == 0:
            continue
        norm = float(r.norm())
        err = float((g - r).norm()) / norm if norm else float(g.abs().max())
        tol = (STATE_TOL if states else TOL)[DTYPES[dtype]]
        log(f"  {n}: {err:.2e} (at most {tol:.2e})")
        assert err <= tol, (n, err, tol)


CASES = [
    # lens, H, G, K, V, init
    ((1,), 2, 2, 64, 64, True),               # a single token
    ((63, 64, 65), 2, 1, 128, 128, False),    # around a tile
    ((31, 32, 33, 1, 0, 130), 3, 3, 128, 64, True),
    ((0, 0, 7, 0), 4, 2, 64, 128, True),      # empty sequences around one
    ((1000,), 2, 1, 64, 64, True),            # one long chain on few heads
    ((257, 5, 640), 6, 2, 128, 128, True),
    ((700, 300), 1, 1, 128, 64, False),
    ((2500, 70, 600), 1, 1, 64, 64, True),    # five runs, one, two
    ((1100, 520), 2, 1, 128, 128, True),
    ((3,) * 40, 16, 4, 64, 64, True),         # many short ones
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,H,G,K,V,init", CASES, ids=lambda v: str(v).replace(" ", "")[:30])
def test_matches_recurrence(ssd, lens, H, G, K, V, init, dtype):
    s = make(lens, H, G, K, V, dtype, seed=sum(lens) + H, init=init)
    log(f"[linattn] {dtype} {lens} H={H} G={G} K={K} V={V}")
    d, ref = on_gpu(s), reference(s)
    check(forward(ssd, d), ref, dtype)
    check(backward(ssd, d), ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decays_from_none_to_no_memory(ssd, dtype):
    """log_decay 0 (a plain sum), about -1e-5, -0.1, -5, -200 (each token for
    itself in 32 bits) and -inf.  The last two leave o_t = scale (q.k) v."""
    decays = [0.0, -1e-5, -0.1, -5.0, -200.0, float("-inf")]
    s = make((150, 400), 6, 6, 64, 64, dtype, seed=5, decays=decays)
    d = on_gpu(s)
    ref = reference(dict(s, ld=torch.tensor(decays[:5] + [-1e30])))
    check(forward(ssd, d), ref, dtype)
    check(backward(ssd, d), ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decays_whose_power_over_a_chunk_is_denormal(ssd, dtype):
    """exp(log_decay) to the power of a chunk's 64 (32) tokens around and below the
    smallest normal fp32 number, 1.2e-38 = e^-87.3."""
    decays = [-1.36, -1.37, -1.5, -1.6, -1.62, -2.7, -2.75, -3.0, -3.2, -3.3]
    s = make((300, 210), 10, 5, 64, 64, dtype, seed=6, decays=decays)
    d, ref = on_gpu(s), reference(s)
    check(forward(ssd, d), ref, dtype)
    check(backward(ssd, d), ref, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_outside_are_neither_read_nor_written(ssd, dtype):
    s = make((70, 0, 200), 4, 2, 128, 64, dtype, seed=9, before=5, after=67)
    d, ref = on_gpu(s), reference(s)
    T, cut = s["q"].shape[0], slice(5, 275)
    dt = DTYPES[dtype]

    def mark(n, size):
        return torch.full((1, T, n, size), 7.0, dtype=dt, device=DEV)

    o, dq, dk, dv = mark(4, 64), mark(2, 128), mark(2, 128), mark(4, 64)
    final, dinit = torch.empty_like(d["init"]), torch.empty_like(d["init"])
    dims = ssd.LinattnDims(T, 3, 4, 2, 128, 64)
    a = (d["q"][None], d["k"][None], d["v"][None], d["ld"], d["init"], d["cu"])
    ws = torch.empty(ssd.linattn_workspace_bytes(dims, dt, True), dtype=torch.uint8, device=DEV)
    ssd.ssd_linattn_fwd(*a, o, final, ws, d["scale"])
    ssd.ssd_linattn_bwd(*a, d["do"][None], d["dfinal"], dq, dk, dv, dinit, ws, d["scale"])
    check({"o": o[0], "final": final, "dq": dq[0], "dk": dk[0], "dv": dv[0], "dinit": dinit},
          ref, dtype, cut)
    for t in (o, dq, dk, dv):
        assert (t[0, :5] == 7).all() and (t[0, 275:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_sequence_of_nan_and_inf_stays_alone(ssd, dtype):
    s = make((66, 90, 33), 2, 2, 64, 64, dtype, seed=11)
    for n in ("q", "k", "v", "do"):
        s[n][66:156] = float("inf") if n == "k" else float("nan")
    s["init"][1] = float("nan")
    s["dfinal"][1] = float("inf")
    d = on_gpu(s)
    got = forward(ssd, d) | backward(ssd, d)
    keep = torch.tensor([t for t in range(189) if not 66 <= t < 156])
    part = dict(s, lens=[66, 33], T=123)
    for n in ("q", "k", "v", "do"):
        part[n] = s[n][keep]
    for n in ("init", "dfinal"):
        part[n] = s[n][[0, 2]]
    got = {n: g.cpu()[[0, 2]] if n in ("final", "dinit") else g.cpu()[keep]
           for n, g in got.items()}
    check(got, reference(part), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_nan_decay_stays_in_its_head(ssd, dtype):
    s = make((150,), 3, 3, 64, 64, dtype, seed=12, decays=[-0.1, float("nan"), -0.1])
    d = on_gpu(s)
    got = forward(ssd, d)
    ref = reference(dict(s, ld=torch.tensor([-0.1, -0.1, -0.1])))
    assert torch.isnan(got["final"][:, 1]).all() and torch.isnan(got["o"][1:, 1]).all()
    keep = [0, 2]
    check({"o": got["o"][:, keep], "final": got["final"][:, keep]},
          {"o": ref["o"][:, keep], "final": ref["final"][:, keep]}, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_batch_form_equals_packed_form(ssd, dtype):
    s = make((150,) * 3, 4, 2, 64, 128, dtype, seed=13)
    d = on_gpu(s)
    packed = forward(ssd, d) | backward(ssd, d)
    b = dict(d, cu=None)
    for n in ("q", "k", "v", "do"):
        b[n] = d[n].view(3, 150, *d[n].shape[1:])
    a = (b["q"], b["k"], b["v"], b["ld"])
    o, final = ssd.linattn(*a, b["init"], None, b["scale"])
    dq, dk, dv, dinit = ssd.linattn_backward(*a, b["do"], b["dfinal"], b["init"], None, b["scale"])
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t.flatten(0, 1), packed[n]), n
    assert torch.equal(final, packed["final"]) and torch.equal(dinit, packed["dinit"])


@pytest.mark.parametrize("lens", [(40,), (900,), (3, 0, 1800), (5000,)])
def test_states_in_place(ssd, lens):
    s = make(lens, 2, 2, 128, 128, "bf16", seed=17)
    d = on_gpu(s)
    want = forward(ssd, d) | backward(ssd, d)
    dims = ssd.LinattnDims(sum(lens), len(lens), 2, 2, 128, 128)
    ws = torch.empty(ssd.linattn_workspace_bytes(dims, torch.bfloat16, True), dtype=torch.uint8,
                     device=DEV)
    a = (d["q"][None], d["k"][None], d["v"][None], d["ld"])
    st = d["init"].clone()
    o = torch.empty_like(d["v"])[None]
    ssd.ssd_linattn_fwd(*a, st, d["cu"], o, st, ws, d["scale"])
    assert torch.equal(st, want["final"]) and torch.equal(o[0], want["o"])
    dq, dk, dv = (torch.empty_like(d[n])[None] for n in ("q", "k", "v"))
    with pytest.raises(ssd.SsdError) as e:      # dk still reads dfinal
        ssd.ssd_linattn_bwd(*a, d["init"], d["cu"], d["do"][None], st, dq, dk, dv, st, ws)
    assert e.value.status == ssd.SSD_ERR_INVALID_ARGUMENT


def test_optional_states_may_be_left_out(ssd):
    s = make((100, 30), 2, 1, 64, 64, "fp32", seed=19, init=False)
    d = on_gpu(s)
    want = forward(ssd, d) | backward(ssd, d)
    dims = ssd.LinattnDims(130, 2, 2, 1, 64, 64)
    ws = torch.empty(ssd.linattn_workspace_bytes(dims, torch.float32, True), dtype=torch.uint8,
                     device=DEV)
    a = (d["q"][None], d["k"][None], d["v"][None], d["ld"], None, d["cu"])
    o = torch.empty_like(d["v"])[None]
    ssd.ssd_linattn_fwd(*a, o, None, ws, d["scale"])
    assert torch.equal(o[0], want["o"])
    dq, dk, dv = (torch.empty_like(d[n])[None] for n in ("q", "k", "v"))
    ssd.ssd_linattn_bwd(*a, d["do"][None], None, dq, dk, dv, None, ws, d["scale"])
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t[0], want[n]), n


def test_gradients_against_differences(ssd):
    """o and final are linear in each of q, k, v and the initial state, so a
    difference of two forward calls is the directional derivative up to fp32
    rounding: of the two calls' outputs, and of sums over them.  Both sides
    are sums of some 1e5 products of size 1 with relative error 64 e each, so
    the difference is below 64 e sqrt(1e5) |f| ~ 1e-3 of their typical size."""
    s = make((90, 45), 2, 1, 64, 64, "fp32", seed=23)
    d = on_gpu(s)
    grads = backward(ssd, d)

    def loss(d):
        f = forward(ssd, d)
        return float((f["o"].double() * d["do"].double()).sum()
                     + (f["final"].double() * d["dfinal"].double()).sum())

    base = loss(d)
    g = torch.Generator().manual_seed(1)
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("init", "dinit")):
        step = torch.randn(d[n].shape, generator=g).to(DEV)
        moved = loss(dict(d, **{n: d[n] + step}))
        want = float((grads[gn].double() * step.double()).sum())
        size = float(grads[gn].double().norm())     # of a directional derivative
        log(f"  {n}: difference {moved - base:.5f} gradient {want:.5f} size {size:.2f}")
        assert abs((moved - base) - want) <= 1e-3 * size


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("b,H,G,K,V", [(1, 1, 1, 64, 64), (1, 2, 1, 128, 128), (3, 24, 8, 64, 128),
                                       (5, 30, 30, 128, 64), (9, 32, 1, 64, 64)])
def test_step_matches_recurrence(ssd, b, H, G, K, V, dtype):
    s = make((1,) * b, H, G, K, V, dtype, seed=b * H)
    d, ref = on_gpu(s), reference(s, backward=False)
    o, state = torch.empty_like(d["v"]), d["init"].clone()
    ssd.ssd_linattn_step(d["q"], d["k"], d["v"], d["ld"], state, o, d["scale"])
    check({"o": o}, ref, dtype)
    # the step's state is one fp32 fma per element, whatever the inputs' type
    err = float((state.double().cpu() - ref["final"]).norm() / ref["final"].norm())
    assert err <= 4 * 2.0 ** -24, err


def test_prompt_then_steps_equal_the_longer_prompt(ssd):
    """A prompt's final state taken on by single tokens: o and the state of
    the sequence that holds them all."""
    s = make((133,), 4, 2, 128, 64, "fp32", seed=29)
    d, ref = on_gpu(s), reference(s, backward=False)
    a = [d[n][None, :130].contiguous() for n in ("q", "k", "v")]
    _, state = ssd.linattn(*a, d["ld"], d["init"], None, d["scale"])
    o = torch.empty_like(d["v"])
    for t in range(130, 133):
        one = [d[n][t:t + 1].contiguous() for n in ("q", "k", "v")]
        out = torch.empty_like(one[2])
        ssd.ssd_linattn_step(*one, d["ld"], state, out, d["scale"])
        o[t] = out[0]
    check({"o": o[130:], "final": state}, {"o": ref["o"][130:], "final": ref["final"]}, "fp32")


@pytest.mark.parametrize("lens", [(70, 5, 40), (1500,)])
def test_captured_and_replayed(ssd, lens):
    """Forward and backward captured into one graph: every replay equals the
    eager call, with other eager work in between."""
    s = make(lens, 4, 2, 64, 64, "bf16", seed=31)
    d = on_gpu(s)
    want = forward(ssd, d) | backward(ssd, d)
    dims = ssd.LinattnDims(sum(lens), len(lens), 4, 2, 64, 64)
    ws = torch.empty(ssd.linattn_workspace_bytes(dims, torch.bfloat16, True), dtype=torch.uint8,
                     device=DEV)
    out = {n: torch.empty_like(t) for n, t in want.items()}
    a = (d["q"][None], d["k"][None], d["v"][None], d["ld"], d["init"], d["cu"])

    def go():
        ssd.ssd_linattn_fwd(*a, out["o"][None], out["final"], ws, d["scale"])
        ssd.ssd_linattn_bwd(*a, d["do"][None], d["dfinal"], out["dq"][None], out["dk"][None],
                            out["dv"][None], out["dinit"], ws, d["scale"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for n, t in out.items():
            assert torch.equal(t, want[n]), n
        again = forward(ssd, d)
        assert torch.equal(again["o"], want["o"])


def test_two_streams_at_once(ssd):
    jobs = [on_gpu(make(lens, 4, 4, 128, 128, "bf16", seed=37 + len(lens)))
            for lens in ((900,), (300, 20, 500))]
    want = [forward(ssd, d) | backward(ssd, d) for d in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        got = []
        for st, d in zip(streams, jobs):
            with torch.cuda.stream(st):
                got.append(forward(ssd, d) | backward(ssd, d))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for n in w:
                assert torch.equal(g[n], w[n]), n


def test_refusals(ssd):
    s = on_gpu(make((10, 6), 4, 2, 64, 64, "bf16", seed=41))
    q, k, v, ld = s["q"][None], s["k"][None], s["v"][None], s["ld"]
    cu = s["cu"]
    with pytest.raises(TypeError):
        ssd.linattn(q, k.float(), v, ld)
    with pytest.raises(TypeError):
        ssd.linattn(q.half(), k.half(), v.half(), ld)
    with pytest.raises(TypeError):
        ssd.linattn(q, k, v, ld, None, cu.long())
    with pytest.raises(ValueError):
        ssd.linattn(q, k[:, :-1].contiguous(), v, ld)
    with pytest.raises(ValueError):
        ssd.linattn(q, k, v, ld[:-1])
    with pytest.raises(ValueError):        # not contiguous
        ssd.linattn(q.transpose(1, 2), k.transpose(1, 2), v, ld)
    with pytest.raises(ValueError):        # states of another number of sequences
        ssd.linattn(q, k, v, ld, s["init"])
    with pytest.raises(ValueError):        # packed sequences in a batch
        ssd.linattn(q.view(2, 8, 2, 64), k.view(2, 8, 2, 64), v.view(2, 8, 4, 64), ld, None, cu)
    with pytest.raises(ValueError):
        ssd.linattn(q, k, v, ld, None, cu.cpu())
    three = v[:, :, :3].contiguous()
    with pytest.raises(ssd.SsdError) as e:  # three heads over two groups
        ssd.linattn(q, k, three, ld[:3].contiguous())
    assert e.value.status == ssd.SSD_ERR_INVALID_ARGUMENT
    odd = [torch.zeros(1, 16, 2, 80, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    with pytest.raises(ssd.SsdError) as e:
        ssd.linattn(*odd, v, ld)
    assert e.value.status == ssd.SSD_ERR_UNSUPPORTED
    ws = torch.empty(8, dtype=torch.uint8, device=DEV)
    with pytest.raises(ssd.SsdError) as e:
        ssd.ssd_linattn_fwd(q, k, v, ld, None, cu, torch.empty_like(v), None, ws)
    assert e.value.status == ssd.SSD_ERR_WORKSPACE


def test_many_sequences_and_heads(ssd):
    """More sequences than a workgroup has threads, many of them empty, and
    enough heads that a sequence is one run."""
    lens = [(7 * i) % 5 if i % 3 else 0 for i in range(700)]
    s = make(lens, 24, 8, 64, 64, "bf16", seed=47)
    d, ref = on_gpu(s), reference(s)
    check(forward(ssd, d), ref, "bf16")
    check(backward(ssd, d), ref, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at,K,V", [(0, 64, 64), (17, 64, 128), (37, 128, 128), (126, 128, 64),
                                    (299, 128, 128)])
def test_a_bad_value_stays_behind_its_token(ssd, dtype, bad, at, K, V):
    """NaN or infinity at one token: every result that has no part of it is as it
    would be without, those of its neighbours in a chunk too."""
    s = make((300,), 4, 2, K, V, dtype, seed=at)
    ref = reference(s)

    def same(got, cut, heads=slice(None), cols=slice(None)):
        for n, g in got.items():
            g, r = g[cut][:, heads, cols].double().cpu(), ref[n][cut][:, heads, cols]
            if r.numel():
                err = float((g - r).norm() / r.norm())
                assert err <= TOL[DTYPES[dtype]], (n, err)

    before, after = slice(0, at), slice(at + 1, 300)
    for name in ("q", "k", "v", "do"):
        x = s[name].clone()
        x[at, 1, 5] = bad
        d = on_gpu(dict(s, **{name: x}))
        fwd, grads = forward(ssd, d), backward(ssd, d)
        o = fwd["o"]
        if name == "v":             # one column of a head's state from that token on
            same({"o": o}, before)
            same({"o": o}, slice(None), slice(2, None))
            same({"o": o}, slice(None), slice(1, 2), slice(6, None))
            assert not torch.isfinite(o[at:, 1, 5]).any()
            final = fwd["final"][0].double().cpu()
            assert not torch.isfinite(final[1, :, 5]).any()
            final[1, :, 5] = ref["final"][0, 1, :, 5]
            err = float((final - ref["final"][0]).norm() / ref["final"].norm())
            assert err <= STATE_TOL[DTYPES[dtype]], err
            same({"dq": grads["dq"]}, before)
            same({"dk": grads["dk"]}, after)
        if name == "k":
            same({"o": o, "dq": grads["dq"]}, before)
            same({"dv": grads["dv"]}, after)
        if name == "q":
            same({"o": o}, before)
            same({"o": o}, after)
            same({"dk": grads["dk"], "dv": grads["dv"]}, after)
        if name == "do":
            same({"dk": grads["dk"], "dv": grads["dv"]}, after)
            same({"dq": grads["dq"]}, before)
            same({"dv": grads["dv"]}, slice(None), slice(1, 2), slice(6, None))


@pytest.mark.parametrize("nseq", [256, 257, 70000])
def test_one_long_sequence_among_many_of_one_token(ssd, nseq):
    """More sequences than a workgroup has threads, and than their square; every
    third is empty, the others have a token, o = scale (q.k) v and k v^T as their
    state, but for one of many runs."""
    at, long, H, K = nseq // 2 // 3 * 3 + 1, 20000, 2, 64
    lens = torch.tensor([i % 3 and 1 for i in range(nseq)])
    lens[at] = long
    cu = torch.zeros(nseq + 1, dtype=torch.int64)
    cu[1:] = lens.cumsum(0)
    T, t0 = int(cu[-1]), int(cu[at])
    g = torch.Generator(device=DEV).manual_seed(nseq)
    q, k, v = (torch.randn(1, T, H, K, generator=g, device=DEV) for _ in range(3))
    ld = torch.tensor([-0.01, -0.3], device=DEV)
    o, final = ssd.linattn(q, k, v, ld, None, cu.to(torch.int32).to(DEV))
    dq, dk, dv, _ = ssd.linattn_backward(q, k, v, ld, v, None, None, cu.to(torch.int32).to(DEV))
    alone = [t[:, t0:t0 + long].contiguous() for t in (q, k, v)]
    lo, lfinal = ssd.linattn(*alone, ld)
    ldq, ldk, ldv, _ = ssd.linattn_backward(*alone, ld, alone[2])
    tol = 2 * TOL[torch.float32]          # (two results with an error each)
    q, k, v = (t[0].double() for t in (q, k, v))
    qk = K ** -0.5 * (q * k).sum(-1, keepdim=True)
    vv = K ** -0.5 * (v * v).sum(-1, keepdim=True)
    for got, one, part in ((o, qk * v, lo), (dq, vv * k, ldq), (dk, vv * q, ldk),
                           (dv, qk * v, ldv)):
        one[t0:t0 + long] = part[0].double()
        err = float((got[0].double() - one).norm() / one.norm())
        assert err <= tol, err
        rest = torch.cat([got[0, :t0], got[0, t0 + long:]]).double()
        one = torch.cat([one[:t0], one[t0 + long:]])
        assert float((rest - one).norm() / one.norm()) <= tol
    idx = torch.nonzero(lens == 1)[:, 0].to(DEV)
    tok = cu.to(DEV)[idx]
    kv = (k[tok, :, :, None] * v[tok, :, None, :]).float()
    assert float((final[idx] - kv).norm() / kv.norm()) <= tol
    assert float((final[at] - lfinal[0]).norm() / lfinal.norm()) <= tol
    assert not final[(lens == 0).nonzero()[:, 0].to(DEV)].any()


def test_bad_offsets_stay_in_range(ssd):
    """Offsets below zero, past the tokens, or descending are taken as the
    nearer end or as empty sequences; sequences that are sound keep their
    results."""
    s = make((40, 60), 2, 2, 64, 64, "fp32", seed=43)
    d = on_gpu(s)
    want = forward(ssd, d)
    d["cu"] = torch.tensor([-5, 40, 4000], dtype=torch.int32, device=DEV)
    got = forward(ssd, d)
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["final"], want["final"])
    d["cu"] = torch.tensor([40, 40, 10], dtype=torch.int32, device=DEV)
    got = forward(ssd, d)                 # two empty ones
    assert torch.equal(got["final"], d["init"])
    # sequences that overlap: any result, but a call that ends, and nothing else hurt
    s = make((3000,), 2, 2, 64, 64, "bf16", seed=44)
    d = on_gpu(s)
    want = forward(ssd, d)
    odd = dict(d, cu=torch.tensor([0, 2900, 100, 3000, 50], dtype=torch.int32, device=DEV),
               init=None, dfinal=None)
    forward(ssd, odd)
    backward(ssd, odd)
    assert torch.equal(forward(ssd, d)["o"], want["o"])


def test_offsets_past_32_bits(ssd):
    """More than 2^31 elements of v, o, dout and dv: the same sequence over and
    over, whose last copy has the first one's results."""
    n, L, H, G, K, V = 132, 1000, 128, 2, 64, 128
    g = torch.Generator(device=DEV).manual_seed(1)

    def rows(heads, size):
        x = torch.randn(1, L, heads, size, generator=g, device=DEV).to(torch.bfloat16)
        return x.expand(n, L, heads, size).contiguous()

    q, k, v, do = rows(G, K), rows(G, K), rows(H, V), rows(H, V)
    assert v.numel() > 2 ** 31
    ld = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H)
    o, final = ssd.linattn(q, k, v, ld)
    grads = ssd.linattn_backward(q, k, v, ld, do)
    one = [t[:1].contiguous() for t in (q, k, v)]
    want_o, want_final = ssd.linattn(*one, ld)
    want = ssd.linattn_backward(*one, ld, do[:1].contiguous())
    # (another number of runs: sums in another order)
    for a, b, dt in ((o, want_o, "bf16"), (final, want_final, "fp32"),
                     *zip(grads, want, ("bf16", "bf16", "bf16", "fp32"))):
        assert torch.equal(a[-1], a[0])
        err = float((a[-1].double() - b[0].double()).norm() / b[0].double().norm())
        assert err <= 2 * max(TOL[DTYPES[dt]], STATE_TOL[DTYPES[dt]]), err
