"""tl_verify_tree: what counts as a probability is the same for a node's first child as for its siblings, in target and draft."""

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
