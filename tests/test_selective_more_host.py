"""Host-side checks of the selective scan (no GPU needed): the comparison of the parameters'
gradients sees sums of fewer bits, and the launch that joins runs has no registers in memory."""
import pytest
import torch

import selective_ref as ref
from test_gpu_selective_sums import SUMS
from test_kernel_scratch_host import scratch  # noqa: F401


def test_sums_in_fewer_bits_are_seen():
    """A mistake planted in the oracle: its sums over tokens kept in 16 significant bits."""
    T, D, N = 3000, 8, 8
    g = torch.Generator().manual_seed(1)
    terms = torch.rand(T, D, N, generator=g, dtype=torch.float64)
    want, low = terms.sum(0), torch.zeros(D, N, dtype=torch.float64)
    for t in range(T):
        part, power = torch.frexp(low + terms[t])
        low = torch.ldexp(torch.round(part * 2.0 ** 16) * 2.0 ** -16, power)
    with pytest.raises(AssertionError):
        ref.check({"dA": low.float()}, {"dA": want}, {"dA": want}, SUMS)
    ref.check({"dA": want.float()}, {"dA": want}, {"dA": want}, SUMS)


def test_scratch_of_the_join(scratch):  # noqa: F811
    sizes = {n: s for n, s in scratch.items() if "scan_join_kernel" in n}
    assert len(sizes) == 4                 # 8, 16, 32 and 64 states
    assert max(sizes.values()) == 0, sizes
