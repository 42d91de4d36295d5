"""Comparison of the linear attention's results head by head, so that a head whose
results are large does not hide another's mistakes.

For each head (dq and dk: group; states: sequence and head) the 2-norm of the error is
at most, with A the norm of the same result of the absolute values of all inputs
(|q|^T sum lam |k| |v|^T and so on: what the products add up to before any cancels),
* bf16 results: 2^-8 of the result (its own rounding, half a step), and (2^-15 + 2^-18) A:
  the scores or the state, and the decayed operand, are two bf16 terms each, which
  leave 2^-16 (half a step, of a remainder of half a step), and fp32 sums as below;
* fp32 results and all states (three terms: exact products): sums of n <= 2^14 fp32
  terms, whose roundings grow like sqrt(n) 2^-24, and decays with a few roundings of
  their own: 2^-16 A.  Up to 1200 terms: 2^-18 A.
Underflow adds to both: a decay, or a term of a split operand, below the smallest normal
number may be lost, 2^-126 of a product of two inputs (below 8 each) at most, three
times in each of up to 2^14 tokens (states), each 2^7 channels long (results):
3 2^(-126 + 6 + 14 + 7) < 2^-97 for each element, times a third input 2^-94."""
import torch

import block_ref

STATES = ("final", "dinit")


def references(q, k, v, log_decay, lens, scale, init=None, do=None, dfinal=None):
    """The 64-bit results, and those of the absolute values."""
    q, k, v = (t.double() for t in (q, k, v))
    do = None if do is None else do.double()
    ref = block_ref.linattn(q, k, v, log_decay, lens, scale, init, do, dfinal)
    init, do, dfinal = (None if t is None else t.abs() for t in (init, do, dfinal))
    size = block_ref.linattn(q.abs(), k.abs(), v.abs(), log_decay, lens, scale, init, do, dfinal)
    return ref, size


def check_heads(got, ref, size, tokens):
    """got: results by name, rows of the packed tokens and states; tokens: of a call."""
    sums = 2.0 ** -18 if tokens <= 1200 else 2.0 ** -16
    worst = {}
    for n, g in got.items():
        g, r, a = g.double().cpu(), ref[n], size[n]
        assert g.shape == r.shape, (n, g.shape, r.shape)
        assert torch.isfinite(g).all(), n
        dims = (-2, -1) if n in STATES else (0, -1)
        err, r, a = (x.square().sum(dims).sqrt() for x in (g - r, r, a))
        if got[n].dtype == torch.bfloat16 and n not in STATES:
            tol = 2.0 ** -8 * r + (2.0 ** -15 + sums) * a
        else:
            tol = sums * a
        tol = tol + 2.0 ** -94 * (g.numel() / max(1, err.numel())) ** 0.5
        worst[n] = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
        bad = (err > tol).nonzero()
        assert bad.numel() == 0, (n, bad[0].tolist(), float(err[tuple(bad[0])]),
                                  float(tol[tuple(bad[0])]))
    return worst
