"""The head-by-head comparison sees a mistake in one quiet head that a norm over all
heads hides: planted in the 64-bit results themselves."""
import pytest
import torch

from block_check import check_heads, references


def results():
    g = torch.Generator().manual_seed(0)
    T, H, K, V = 200, 3, 64, 64
    q, k, v, do = (torch.randn(T, H, d, generator=g).double() for d in (K, K, V, V))
    init, dfinal = (torch.randn(1, H, K, V, generator=g).double() for _ in range(2))
    ld = torch.tensor([0.0, -0.1, -5.0])
    return references(q, k, v, ld, [T], K ** -0.5, init, do, dfinal)


@pytest.mark.parametrize("name", ["o", "dq", "dk", "dv", "final", "dinit"])
def test_a_mistake_in_a_quiet_head_is_seen(name):
    ref, size = results()
    good = {n: (x if n in ("final", "dinit") else x.bfloat16()) for n, x in ref.items()}
    check_heads(good, ref, size, 200)
    bad = dict(good, **{name: good[name].clone()})
    bad[name][:, -1] *= 1.02           # states: a sequence's head; rows: every token's head
    err = float((bad[name].double() - ref[name]).norm() / ref[name].norm())
    assert name in ("final", "dinit") or err < 2.0 ** -8, err   # what one norm says of it
    with pytest.raises(AssertionError):
        check_heads(bad, ref, size, 200)
