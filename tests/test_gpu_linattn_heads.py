"""Linear attention head by head (block_check.py has the tolerances): decays from none
to no memory, whose large heads would hide the others in one norm over all of them,
powers of decays around the smallest normal number, and ragged sequences."""
import pytest
import torch

from block_check import check_heads, references
from gpu_util import log
from test_gpu_linattn import CASES, backward, forward, make, on_gpu, ssd  # noqa: F401

pytestmark = pytest.mark.gpu

DECAYS = [
    [0.0, -1e-5, -0.1, -5.0, -200.0, float("-inf")],
    [-1.36, -1.37, -1.5, -1.6, -1.62, -2.7, -2.75, -3.0, -3.2, -3.3],
    [-20.0, -0.3, -0.01, -87.0],
]


def run(ssd, s, what):
    cut = slice(s["before"], s["before"] + s["T"])
    ld = s["ld"].clamp(min=-1e30)
    ref, size = references(*(s[n][cut] for n in ("q", "k", "v")), ld, s["lens"], s["scale"],
                           s["init"], s["do"][cut], s["dfinal"])
    d = on_gpu(s)
    worst = check_heads(forward(ssd, d) | backward(ssd, d), ref, size, s["T"])
    log(f"  {what}: of the tolerance " + ", ".join(f"{n} {w:.2f}" for n, w in worst.items()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("decays", DECAYS, ids=["wide", "denormal", "mixed"])
def test_each_decay_by_itself(ssd, decays, K, V, dtype):  # noqa: F811
    H = len(decays)
    s = make((150, 400, 77), H, H if K == V else H // 2, K, V, dtype, seed=K + 2 * V + H,
             decays=decays)
    run(ssd, s, f"{dtype} {K}x{V}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,H,G,K,V,init", CASES, ids=lambda v: str(v).replace(" ", "")[:30])
def test_each_head_by_itself(ssd, lens, H, G, K, V, init, dtype):  # noqa: F811
    s = make(lens, H, G, K, V, dtype, seed=sum(lens) + 2 * H, init=init)
    run(ssd, s, f"{dtype} {lens}")


@pytest.mark.parametrize("G,H", [(2, 4), (3, 3)])
def test_equal_lengths_are_the_ssd_with_constant_steps(ssd, G, H):  # noqa: F811
    """x = v, B = k, C = scale q, dt = 1, A = log_decay, D = 0; and a further token on the
    transposed state.  fp32: each side as far from exact as the parity tests allow, 1e-4
    of the largest of a value and the root mean square."""
    b, L, K, V = 2, 150, 128, 64
    g = torch.Generator().manual_seed(G)
    q, k = (torch.randn(b, L, G, K, generator=g).to("cuda:0") for _ in range(2))
    v = torch.randn(b, L, H, V, generator=g).to("cuda:0")
    ld = -torch.rand(H, generator=g).to("cuda:0")
    scale, ones, none = K ** -0.5, torch.ones(b, L, H, device="cuda:0"), torch.zeros_like(ld)
    o, final = ssd.linattn(q, k, v, ld)
    y, _, last = ssd.forward(v, ones, ld, k, q * scale, none)

    def close(a, r):
        assert float((a - r).abs().max() / r.square().mean().sqrt()) <= 2e-4

    close(o, y)
    close(final.transpose(-1, -2), last)
    q1, k1, v1 = (t[:, 0].contiguous() for t in (q, k, v))
    o1, y1 = torch.empty_like(v1), torch.empty_like(v1)
    ssd.ssd_linattn_step(q1, k1, v1, ld, final, o1)
    ssd.ssd_decode_step(v1, ones[:, 0].contiguous(), ld, k1, q1 * scale, none, last, y1)
    close(o1, y1)
    close(final.transpose(-1, -2), last)
