"""The gradients of the parameters (A, D and the bias of dt) are sums over all tokens held in 32
bits: their errors are those of 32 bits, which sums of fewer bits would exceed.

Tolerance.  A token's term is a product of R, h, a decay and the time step.  R and h are sums over
the tokens that a state remembers, here (time steps of some 0.7, A of -1 and less) two on
average and 30 at most, and each token's decay, sum and time step are good to 2^-22 together: a
term is good to sqrt(30) 2^-22 < 2^-19.5 of its sum of absolute values, and those of different
tokens do not agree in sign.  Sums over a run (144 tokens at most) and over the runs are good to
sqrt(144) 2^-25 + 2^-24 < 2^-21.  2^-19 of the sum of absolute values, channel by channel; a sum in
bf16 with its 2^-9 a step, or in 16 significant bits (2^-17 a step), lies far outside."""
import pytest
import torch

import selective_ref as ref
from selective_util import DEV

pytestmark = pytest.mark.gpu
SUMS = 2.0 ** -19


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


@pytest.mark.parametrize("N,G,lens", [(16, 1, [3000]), (8, 2, [1100, 1, 0, 1200, 700]),
                                      (32, 1, [1500, 900]), (64, 1, [1000])])
def test_sums_over_tokens(ssd, N, G, lens):
    D, T = 48, sum(lens)
    g = torch.Generator().manual_seed(N)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    # one sign for what the sums are over, so that they grow with the tokens
    x, B, C, dy = (t.abs() for t in (normal(T, D), normal(T, G, N), normal(T, G, N), normal(T, D)))
    z, dt = normal(T, D).abs() + 0.5, normal(T, D) * 0.3
    A = -torch.arange(1, N + 1).float() * (1 + 0.2 * normal(D, N)).abs() - 0.1
    skip, bias = normal(D), normal(D) * 0.1
    args = [t.double() for t in (x, dt, A, B, C, skip, z, bias)]
    want = ref.scan(*args, lens, True, None, dy.double())
    size = ref.scan(*args, lens, True, None, dy.double(), size=True)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    rows = [t[None].to(DEV) for t in (x, dt, B, C, z, dy)]
    grads = ssd.selective_scan_backward(rows[0], rows[1], A.to(DEV), rows[2], rows[3],
                                        skip.to(DEV), rows[4], bias.to(DEV), rows[5], None, None, cu)
    got = {"dA": grads[2], "dD": grads[5], "ddt_bias": grads[7]}
    worst = ref.check(got, want, size, SUMS)
    print({n: round(v, 4) for n, v in worst.items()})
