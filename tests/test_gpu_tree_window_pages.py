"""tl_tree_attention under a window: pages that no node sees a key of need not exist."""

import numpy as np
import pytest
import torch

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_tree_attention import attend, case, compare

pytestmark = pytest.mark.gpu


def seen_pages(words, starts, lens, b, page, window, sinks):
    """Pages of request b with a key that one of its nodes sees; its nodes' own places are always cached."""
    n = int(starts[b + 1] - starts[b])
    keys = set(range(lens[b], lens[b] + n))
    for t in range(starts[b], starts[b + 1]):
        keys |= set(O.tree_seen(lens[b], words[t] & ((1 << n) - 1), window, sinks))
    return {k // page for k in keys}


def without_the_others(table, words, starts, lens, page, window, sinks, bad):
    t = table.copy()
    for b in range(len(lens)):
        keep = seen_pages(words, starts, lens, b, page, window, sinks)
        t[b, [i for i in range(t.shape[1]) if i not in keep]] = bad
    return t


@pytest.mark.parametrize("page", [1, 7, 16, 32])
@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 20), (97, 3)])
@pytest.mark.parametrize("d,cache", [(64, "bf16"), (128, "f8"), (256, "f16")])
def test_only_pages_that_a_node_sees(page, window, sinks, d, cache):
    """Lengths around a page's border, so that the window begins at one; a node alone, trees, and chains of which the first node sees most."""
    lens = [window + 5 * page + i for i in (-1, 0, 1, page // 2)] + [window - 1, window, window + 1, 3, 3 * window + 200]
    nodes = [1, 1, 5, 1, 1, 3, 1, 2, 64]
    kv, q, words, starts, table, k64, v64 = case(page + window, lens, nodes, 6, 2, d, page, cache)
    spare = int(np.setdiff1d(np.arange(kv.num_pages), table)[0])               # holds NaN
    for bad in (-1, 1 << 30, spare):
        t = without_the_others(table, words, starts, lens, page, window, sinks, bad)
        assert np.any(t[:, 0] == bad) == (sinks == 0)             # (the input is what it is meant to be)
        out, lse = attend(kv, q, words, starts, t, lens, window=window, sinks=sinks)
        assert tl.tl_get_status() == tl.TL_OK
        compare(out, lse, q, words, starts, table, k64, v64, lens, window, sinks)


@pytest.mark.parametrize("page", [7, 16])
def test_masks_of_any_bits(page):
    """The window counts a mask's bits: none at all leaves it `window` cached tokens, many leave few; what the row with the fewest sees is needed."""
    window, lens, nodes = 80, [400, 401, 402, 403, 300], [3, 64, 40, 2, 9]
    rng = np.random.default_rng(page)
    starts = np.concatenate([[0], np.cumsum(nodes)])
    words = [int(w) for w in rng.integers(0, 1 << 63, sum(nodes), dtype=np.uint64)]
    words[0:3] = [0, 7, 3]                                       # the first request has a row without nodes
    words[3:67] = [(1 << 64) - 1 - (1 << i) for i in range(64)]  # the second sees 63 nodes everywhere: 17 cached tokens
    kv, q, words, starts, table, k64, v64 = case(31, lens, nodes, 4, 2, 64, page, masks=words)
    t = without_the_others(table, words, starts, lens, page, window, 0, -1)
    assert t[1, (401 - 18) // page - 1] == -1 and t[0, (400 - 80) // page] != -1
    out, lse = attend(kv, q, words, starts, t, lens, window=window)
    assert tl.tl_get_status() == tl.TL_OK
    compare(out, lse, q, words, starts, table, k64, v64, lens, window)
    for b in range(len(lens)):                                   # and each of those that are left is looked at
        for i in np.flatnonzero(t[b] >= 0):
            if i * page < lens[b] + nodes[b]:
                worse = t.copy()
                worse[b, i] = -1
                attend(kv, q, words, starts, worse, lens, window=window)
                assert tl.tl_get_status() == tl.TL_EDATA, (b, int(i))


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_a_tree_of_one_node_takes_the_table_of_its_decode_step(cache):
    window, page = 64, 16
    lens = list(range(window + 40, window + 40 + 2 * page))
    kv, q, words, starts, table, k64, v64 = case(33, lens, [1] * len(lens), 4, 2, 128, page, cache)
    t = table.copy()
    for b, n in enumerate(lens):
        t[b, :(n + 1 - window) // page] = -1
    step = kv.attend(q.cuda(), torch.tensor(t).cuda(), torch.tensor([n + 1 for n in lens], dtype=torch.int32).cuda(), window=window).double()
    assert tl.tl_get_status() == tl.TL_OK
    out, _ = attend(kv, q, words, starts, t, lens, window=window)
    assert tl.tl_get_status() == tl.TL_OK
    assert torch.all((out.double() - step).abs() <= 2.0 ** -7 * step.abs() + 2.0 ** -14)      # both rounded to bf16
