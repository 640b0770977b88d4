"""Trees of drafted tokens: rows before the first request are padding, as those behind the last are."""

import numpy as np
import pytest
import torch

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_tree import dev

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
