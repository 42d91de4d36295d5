"""The selective scan and its gradients where decays are larger than 1, up to products of 2^100
over a sequence, against the 64-bit recurrence.

Tolerance (selective_ref.check): none of the tokens is forgotten, and equal time steps round alike,
so the errors of a product add up.  Its exponents' sum is at most 68 (0.17 times 400), with three
roundings of 2^-24 each: 2^-16.3; 400 exponentials are good to 2^-23 each: 2^-14.4.  With a state's
own roundings (sqrt(400) 2^-24) below 2^-13.9; 2^-13.5 of the sum of absolute values."""
import pytest
import torch

import selective_ref as ref
from selective_util import DEV, dbl

pytestmark = pytest.mark.gpu
SUMS = 2.0 ** -13.5


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


@pytest.mark.parametrize("T,top,softplus", [(20, 0.3, True), (400, 0.17, True),
                                            (400, 0.17, False)])
def test_decays_larger_than_one(ssd, T, top, softplus):
    D, N = 96, 16
    g = torch.Generator().manual_seed(T)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    x, z, dy, B, C = normal(T, D), normal(T, D), normal(T, D), normal(T, 1, N), normal(T, 1, N)
    if softplus:
        # time steps of 0.7 (the logarithm of 2), an exponent of at most `top` a token
        dt, A = torch.zeros(T, D), torch.rand(D, N, generator=g) * top / 0.7
    else:
        dt, A = torch.rand(T, D, generator=g) - 1.0, -torch.rand(D, N, generator=g) * top
    A[:, 0] = -1.0 if softplus else 1.0
    skip, init, dfinal = normal(D), normal(1, D, N), normal(1, D, N)
    args = [t.double() for t in (x, dt, A, B, C, skip, z)]
    args += [None, [T], softplus, init.double(), dy.double(), dfinal.double()]
    want, size = ref.scan(*args), ref.scan(*args, size=True)
    assert want["final"].abs().max() > (100.0 if T == 20 else 1e15)
    x, dt, z, dy, B, C = (t[None].to(DEV) for t in (x, dt, z, dy, B, C))
    ins = (x, dt, A.to(DEV), B, C, skip.to(DEV), z, None)
    y, final = ssd.selective_scan(*ins, init.to(DEV), None, softplus)
    grads = ssd.selective_scan_backward(*ins, dy, dfinal.to(DEV), init.to(DEV), None, softplus)
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit")
    got = {"y": y, "final": final, **dict(zip(names, grads))}
    del got["ddt_bias"]
    got = {n: t[0] if n in ("y", "dx", "ddt", "dB", "dC", "dz") else t for n, t in got.items()}
    worst = ref.check(got, want, size, SUMS)
    print({n: round(v, 3) for n, v in worst.items()}, float(dbl(final).abs().max()))
