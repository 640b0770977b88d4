"""Trees of drafted tokens: rows of no request are padding wherever they lie, and append stores nothing of them."""

import numpy as np
import pytest
import torch

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_tree import dev, draws, expected

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def planned(kv, parents, starts, lens, pages):
    """With outputs that hold a place of the cache beforehand."""
    T = len(parents)
    got = [torch.full((T,), 5, dtype=t, device="cuda") for t in (I64, I32, I64)]
    kv.plan_tree(dev(parents, I32), dev(starts, I32), dev(lens, I32), dev(np.array(pages).reshape(len(lens), -1), I32), *got)
    return [x.tolist() for x in got]


@pytest.mark.parametrize("before,behind", [(3, 0), (1, 2), (100, 70), (5, 0)])
def test_plan_of_rows_before_the_first_request(before, behind):
    kv = tl.PagedKVCache(4, 16, 1, 16)
    parents = [7] * before + [-1, 0, 0, -1, 0] + [7] * behind
    masks, positions, slots = planned(kv, parents, [before, before + 3, before + 5], [4, 30], [[0, 1], [2, 3]])
    assert tl.tl_get_status() == tl.TL_OK
    assert masks == [0] * before + [1, 3, 5, 1, 3] + [0] * behind
    assert positions == [0] * before + [4, 5, 5, 30, 31] + [0] * behind
    assert slots == [-1] * before + [4, 5, 6, 32 + 30, 32 + 31] + [-1] * behind


def test_plan_without_requests():
    kv = tl.PagedKVCache(4, 16, 1, 16)
    for start in (0, 3, 6):
        got = [torch.full((6,), 5, dtype=t, device="cuda") for t in (I64, I32, I64)]
        kv.plan_tree(dev([-1] * 6, I32), dev([start], I32), dev(np.zeros(0), I32), torch.zeros((0, 2), dtype=I32, device="cuda"), *got)
        assert tl.tl_get_status() == tl.TL_OK and [x.tolist() for x in got] == [[0] * 6, [0] * 6, [-1] * 6]


@pytest.mark.parametrize("before,behind", [(3, 0), (1, 2), (300, 70)])
def test_verification_of_rows_before_the_first_request(before, behind):
    rng = np.random.default_rng(before)
    nodes = [4, 1, 9]
    parents, target, draft, tokens, uniform = draws(rng, nodes, 300)
    T, total = sum(nodes), before + sum(nodes) + behind

    def rows(x, fill):
        x = np.asarray(x)
        full = np.full((total,) + x.shape[1:], fill, dtype=x.dtype)
        full[before:before + T] = x
        return dev(full)

    path = torch.full((total,), 5, dtype=I32, device="cuda")
    starts = before + np.concatenate([[0], np.cumsum(nodes)])
    _, counts, after = tl.tl_verify_tree(rows(target, np.nan), rows(draft, np.nan), rows(tokens.astype(np.int32), 7), rows(np.array(sum(parents, []), dtype=np.int32), 7),
                                         dev(starts, I32), rows(uniform, 0), path=path)
    want = expected(parents, target, draft, tokens, uniform, nodes, pad=behind)
    assert tl.tl_get_status() == tl.TL_OK
    assert [path.tolist(), counts.tolist(), after.tolist()] == [[-1] * before + want[0]] + want[1:]


def test_verification_of_requests_out_of_order():
    """The first request's start lies behind the second's rows: only those before all of them are padding."""
    rng = np.random.default_rng(2)
    parents, target, draft, tokens, uniform = draws(rng, [9], 300)
    full = [np.concatenate([np.repeat(x[:1], 3, 0), x, np.repeat(x[:1], 4, 0)]) for x in (target, draft, tokens, np.array(parents[0], dtype=np.int32), uniform)]
    path = torch.full((16,), 5, dtype=I32, device="cuda")
    t, d, k, p, u = (dev(x) for x in full)
    _, counts, after = tl.tl_verify_tree(t, d, k.int(), p.int(), dev([7, 3, 12], I32), u, path=path)
    want = expected(parents, target, draft, tokens, uniform, [9])
    assert tl.tl_get_status() == tl.TL_EDATA
    assert [path[:12].tolist(), counts.tolist(), after.tolist()] == [[-1] * 3 + want[0], [0] + want[1], [-1] + want[2]]


@pytest.mark.parametrize("starts,lens", [([0, 65, 70], [4, 9]), ([0, 90, 70], [4, 9]), ([-3, 65, 70], [4, 9]), ([0, 3, 99], [4, 9]), ([0, 3, 71], [4, 9]),
                                         ([99, 3, 70], [4, 9]), ([99, 3, 40], [4, 9]), ([50, 3, 60], [4, 9]), ([0, 3, -1], [4, 9]), ([-5, -9, -1], [4, 9]),
                                         ([0, 3, 67], [-1, 9]), ([0, 3, 67], [2 ** 31 - 1, 9]), ([0, 3, 67], [4, 97])])
def test_a_refused_request_has_no_places(starts, lens):
    """What append would store somewhere is left of its rows: nothing that lies there by chance."""
    kv = tl.PagedKVCache(12, 16, 1, 16)
    pages = [[11, 10, 9, 8, 7, 6], [0, 1, 2, 3, 4, 5]]
    _, _, slots = planned(kv, [-1] * 70, starts, lens, pages)
    assert tl.tl_get_status() == tl.TL_EDATA
    of = [-1] * 70                                               # who has a row, as far as that is said
    for b in range(2):
        if 0 <= starts[b] <= starts[b + 1] <= 70 and starts[b + 1] - starts[b] <= 64:
            of[starts[b]:starts[b + 1]] = [b] * (starts[b + 1] - starts[b])
    for t, b in enumerate(of):
        place = lens[b] + t - starts[b]
        fits = b >= 0 and 0 <= lens[b] <= 96 - (starts[b + 1] - starts[b])
        assert slots[t] == (pages[b][place // 16] * 16 + place % 16 if fits else -1), t
