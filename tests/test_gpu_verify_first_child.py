"""tl_verify_tree: what counts as a probability is the same for a node's first child as for its siblings, in target and draft."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_tree import verified

pytestmark = pytest.mark.gpu

NAN, INF, BELOW = float("nan"), float("inf"), 1 - 2.0 ** -24
# target's and draft's probability of the child's token, and its uniform number
ODD = [(0.0, -0.1, 0.5), (0.25, NAN, 0.5), (0.25, NAN, BELOW), (1.0, 2.0, 0.7), (1.0, 1.0000001, BELOW), (NAN, -0.1, 0.5), (NAN, NAN, 0.0),
       (-0.5, -1.0, 0.9), (0.0, -INF, 0.9), (INF, INF, 0.5), (INF, 0.5, 0.9), (1.5, 1.25, BELOW), (0.5, INF, 0.6), (0.5, INF, 0.4), (0.25, -3.0, 0.9)]


@pytest.mark.parametrize("p,q,u", ODD)
@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("vocab", [6, 40000])
def test_below_zero_nan_and_above_one(p, q, u, second, vocab):
    target, draft = np.zeros((3, vocab), dtype=np.float32), np.zeros((3, vocab), dtype=np.float32)
    target[0, [2, vocab - 1]] = p, 0.0 if p >= 1 else 0.3
    draft[0, [2, 4]] = q, 0.1
    target[1:, 1] = draft[1:, 1] = 1
    parents, tokens = ([-1, 0, 0], [0, 4, 2]) if second else ([-1, 0, 1], [0, 2, 1])      # token 4: never the target's
    uniform = np.array([0.5, 0.5 if second else u, u if second else 0.0], dtype=np.float32)
    plain = [np.clip(np.nan_to_num(x, nan=0.0, posinf=1.0, neginf=0.0), 0, 1) for x in (target, draft)]
    way, after = O.verify_tree(*plain, tokens, parents, uniform)
    assert verified([parents], target, draft, np.array(tokens, dtype=np.int32), uniform, [3]) == [way + [-1] * (3 - len(way)), [len(way)], [after]]
    assert tl.tl_get_status() == tl.TL_OK


def test_products_at_the_border_exactly():
    """u q < p of a first child, where u q and p agree to all bits of a float or nearly, subnormal numbers among them."""
    rng = np.random.default_rng(0)
    n = 3000
    q = np.float32(2) ** rng.uniform(-148.9, 0, n).astype(np.float32)
    u = rng.random(n).astype(np.float32)
    u[::3] = BELOW
    p = (u.astype(np.float64) * q).astype(np.float32)           # (48 bits: exact in 64-bit floats, rounded once)
    p[::7] = np.nextafter(p[::7], np.float32(0))
    p[::11] = np.nextafter(p[::11], np.float32(1))
    u[:4], q[:4], p[:4] = [BELOW] * 4, [1e-40, 1e-40, 2.0 ** -149, 2.0 ** -149], [1e-40, 1e-40 - 2.0 ** -149, 2.0 ** -149, 0.0]
    target, draft = np.zeros((2 * n, 4), dtype=np.float32), np.zeros((2 * n, 4), dtype=np.float32)
    target[::2, 2], draft[::2, 2], target[1::2, 1] = p, q, 1
    tokens, uniform = np.tile([0, 2], n).astype(np.int32), np.zeros(2 * n, dtype=np.float32)
    uniform[1::2] = u
    want = [2 if Fraction(float(a)) * Fraction(float(b)) < Fraction(float(c)) else 1 for a, b, c in zip(u, q, p)]
    assert {1, 2} == set(want[4:]) and want[:4] == [2, 1, 2, 1]
    assert verified([[-1, 0]] * n, target, draft, tokens, uniform, [2] * n)[1] == want
    assert tl.tl_get_status() == tl.TL_OK
