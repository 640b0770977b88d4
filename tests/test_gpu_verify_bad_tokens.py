"""tl_verify_tree: a guess outside the vocabulary is a refused one. It is one token more, which neither distribution gives any probability."""

import numpy as np
import pytest

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_tree import draws, expected, verified

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [5, 1000, 40001])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("chain", [True, False])
def test_tokens_outside_the_vocabulary(vocab, drafted, chain):
    rng = np.random.default_rng(vocab + drafted)
    nodes = [8, 1, 30, 2, 64, 20]
    parents, target, draft, tokens, uniform = draws(rng, nodes, vocab, drafted, chain, near=0.6)
    out = rng.random(len(tokens)) < 0.35
    more = lambda x: None if x is None else np.pad(x, ((0, 0), (0, 1)))      # noqa: E731
    want = expected(parents, more(target), more(draft), np.where(out, vocab, tokens), uniform, nodes)
    for bad in (vocab, -1, 2 ** 31 - 1, -2 ** 31):
        got = verified(parents, target, draft, np.where(out, bad, tokens).astype(np.int64), uniform, nodes)
        assert tl.tl_get_status() == tl.TL_EDATA
        assert got == want


@pytest.mark.parametrize("drafted", [True, False])
def test_siblings_of_such_a_token(drafted):
    """What is left to the later ones, and to the token after, is what a refusal leaves."""
    f = np.float32
    target = np.array([[.4, .3, .2, .1]] * 4, dtype=f)
    draft = np.array([[.1, .2, .3, .4]] * 4, dtype=f)
    for first in (-1, 4):
        for u in (.05, .3, .45, .6, .9):
            tokens = np.array([0, first, 0, 1])
            uniform = np.array([.55, 0, u, u], dtype=f)
            more = lambda x: np.pad(x, ((0, 0), (0, 1)))         # noqa: E731
            want = expected([[-1, 0, 0, 0]], more(target), more(draft) if drafted else None, np.array([0, 4, 0, 1]), uniform, [4])
            assert verified([[-1, 0, 0, 0]], target, draft if drafted else None, tokens, uniform, [4]) == want
            assert tl.tl_get_status() == tl.TL_EDATA
