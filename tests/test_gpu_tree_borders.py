"""The token that tl_verify_tree draws, at the borders between tokens.

What is left after refusals is worked out in exact rational numbers, and the uniform number is the float nearest to a border of the tokens,
of all borders the one that is met best. The documentation promises 44 bits of sums and differences; with up to 4 refusals and their
multiples a border is moved by 8 2^-44 of one at most, so those further than 2^-40 from the float have to decide as they exactly do."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("refused", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("vocab", [700, 5000, 20000])
@pytest.mark.parametrize("drafted", [True, False])
def test_tokens_at_their_borders(vocab, refused, drafted):
    rng = np.random.default_rng(vocab + refused)
    n = 1 + refused

    def row(sharp):
        e = np.exp(sharp * rng.standard_normal(vocab))
        return (e / e.sum()).astype(np.float32)

    p = row(1.0)
    q = (0.6 * p + 0.4 * row(1.0)).astype(np.float32)
    # refused children: tokens of which the draft thinks more than the target (chosen ones: the number decides, u = 1 - 2^-24 above p)
    likely = np.flatnonzero(q > p) if drafted else np.arange(vocab)
    tokens = np.concatenate([[0], rng.choice(likely, refused, replace=False)]).astype(np.int32)
    uniform = np.full(n, 1 - 2.0 ** -24, dtype=np.float32)

    one = 1 << 160                                     # every float here is a multiple of 2^-149
    left = [int(Fraction(float(x)) * one) for x in p]
    prob = [int(Fraction(float(x)) * one) for x in q]
    s = one
    for c in tokens[1:]:
        if drafted:
            if s == one:
                left = [max(a - b, 0) for a, b in zip(left, prob)]
            else:                                      # (floor of 2^-160: nothing here)
                left = [max(a - s * b // one, 0) for a, b in zip(left, prob)]
        else:
            left[c] = 0
        s = sum(left)
    total = sum(left)
    best, run, at = None, 0, None
    for x in range(vocab - 1):
        run += left[x]
        if left[x] == 0:
            continue
        exact = Fraction(run, total)
        u = np.float32(float(exact))
        off = abs(Fraction(float(u)) * total - run) / one
        if off > Fraction(1, 1 << 40) and float(u) < 1 and (best is None or off < best):
            best, at = off, u
    assert best < Fraction(1, 1 << 30)                 # (the input is what it is meant to be)
    uniform[0] = at
    goal, run, want = Fraction(float(at)) * total, 0, None
    for x in range(vocab):
        run += left[x]
        if run > goal:
            want = x
            break
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()      # noqa: E731
    rows = lambda a: dev(np.tile(a, (n, 1)))                               # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")      # noqa: E731
    path, counts, after = tl.tl_verify_tree(rows(p), rows(q) if drafted else None, dev(tokens), i32([-1] + [0] * refused), i32([0, n]), dev(uniform))
    assert tl.tl_get_status() == tl.TL_OK
    assert counts.tolist() == [1] and path.tolist() == [0] + [-1] * refused
    assert after.tolist() == [want], float(best)
