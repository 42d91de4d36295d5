"""The selective scan's form for single tokens with and without softplus, and with the skip, the
gate and the bias each alone, against the 64-bit recurrence.

Tolerance (selective_ref.check): one token's state and output have an exponential good to 2^-23,
a time step good to some 2^-22 and sums of at most 66 terms: 2^-20 of the sum of absolute values,
plus y's own rounding.  Without softplus some time steps are negative: exponents delta A reach 19.5 for
these inputs, where no decay makes up for the roundings of the time step, of log2(e) and of their
two products, 2^-24 of the exponent or less each: 19.5 * 4 * 2^-24 = 2^-17.7; 2^-17 there."""
import itertools

import pytest
import torch

import selective_ref as ref
from selective_util import DEV, TYPES, Guarded, dbl, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


OPTIONS = list(itertools.product([True, False], repeat=3))       # D, z, dt_bias


@pytest.mark.parametrize("D,z,bias", OPTIONS)
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("b,dim,N,G,dt", [(3, 96, 16, 2, "bf16"), (5, 33, 64, 3, "fp32")])
def test_step(ssd, b, dim, N, G, dt, softplus, D, z, bias):
    g = torch.Generator().manual_seed(b * 8 + 4 * D + 2 * z + bias)
    dt = TYPES[dt]

    def rows(*shape, std=1.0, offset=0.0):
        return (torch.randn(b, *shape, generator=g) * std + offset).to(dt).to(DEV)

    # (without softplus time steps are what they are; some are negative)
    de = rows(dim, std=0.7) if softplus else rows(dim, std=0.1, offset=0.1)
    x, B, C, gate = rows(dim), rows(G, N), rows(G, N), rows(dim)
    A = -torch.rand(dim, N, generator=g) * N
    skip, shift = torch.randn(dim, generator=g), torch.randn(dim, generator=g) * 0.1
    state = torch.randn(b, dim, N, generator=g)
    gate, skip, shift = (t if on else None for t, on in ((gate, z), (skip, D), (shift, bias)))
    args = (dbl(x), dbl(de), A.double(), dbl(B), dbl(C), dbl(skip), dbl(gate), dbl(shift), [1] * b,
            softplus, state.double())
    want, size = ref.scan(*args), ref.scan(*args, size=True)
    out = Guarded()
    y, s = out((b, dim), dt), out((b, dim, N), torch.float32)
    s.copy_(state)
    ssd.ssd_selective_scan_step(x, de, dev(A), B, C, dev(skip), gate, dev(shift), s, y, softplus)
    out.check()
    ref.check({"y": y, "final": s}, want, size, 2.0 ** -20 if softplus else 2.0 ** -17)
