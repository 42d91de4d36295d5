"""Linear attention where the products with the state cancel: the summed operands
share a mean, the other one sums to zero over its channels, so an output is a
small difference of large products and shows how the state is held.

With A the same recurrence on absolute values (|q|^T sum lam |k| |v|^T and so on),
the bf16 walks differ from the exact result by at most
* 2^-8 of the output (its own rounding, half a step);
* 2^-16 A for the state and 2^-16 A for the decayed operand added to it, each as two
  bf16 terms (half a step, of a remainder of half a step); the scores' two terms
  fall on the products within a chunk, which are not in the state;
* fp32 sums of up to n = 1200 products: sqrt(n) 2^-24 A < 2^-18 A.
The test takes the 2-norms of both sides, for each head (or group) alone.  One
bf16 term for the state would leave 2^-8 A, some hundred times the second bound.
"""
import pytest
import torch

import block_ref
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_chunked_fwd_amd as m
    return m


@pytest.mark.parametrize("out,centred", [("o", "q"), ("dq", "do"), ("dk", "v"), ("dv", "k")])
@pytest.mark.parametrize("lens,H,G,K,V", [((1000,), 2, 1, 128, 128), ((700, 150), 3, 3, 128, 64),
                                          ((1100,), 2, 2, 64, 128), ((600, 64, 1), 4, 2, 64, 64)])
def test_products_that_cancel(ssd, lens, H, G, K, V, out, centred):
    g = torch.Generator().manual_seed(sum(lens) + K + V)
    T = sum(lens)
    s = {}
    for n, heads, size in (("q", G, K), ("k", G, K), ("v", H, V), ("do", H, V)):
        x = torch.randn(T, heads, size, generator=g)
        x = x - x.mean(-1, keepdim=True) if n == centred else 1 + 0.3 * x
        s[n] = x.to(torch.bfloat16)
    ld = -torch.logspace(-3, -2, H)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    q, k, v, do = (s[n][None].to(DEV) for n in ("q", "k", "v", "do"))
    if out == "o":
        got = ssd.linattn(q, k, v, ld.to(DEV), None, cu)[0]
    else:
        got = ssd.linattn_backward(q, k, v, ld.to(DEV), do, None, None, cu)
        got = dict(zip(("dq", "dk", "dv"), got))[out]
    q, k, v, do = (s[n].double() for n in ("q", "k", "v", "do"))
    ref = block_ref.linattn(q, k, v, ld, lens, K ** -0.5, do=do)[out]
    size = block_ref.linattn(q.abs(), k.abs(), v.abs(), ld, lens, K ** -0.5, do=do.abs())[out]
    got = got[0].double().cpu()
    for h in range(ref.shape[1]):
        err, r, a = (float(x[:, h].norm()) for x in (got - ref, ref, size))
        log(f"  {out} head {h}: {err / r:.2e} of the output, products {a / r:.0f} times it")
        assert err <= 2.0 ** -8 * r + (2.0 ** -15 + 2.0 ** -18) * a, (out, h, err / r)
