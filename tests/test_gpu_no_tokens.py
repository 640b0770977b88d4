"""Calls without tokens or requests do nothing, whatever the strides of their empty tensors."""

import numpy as np
import pytest
import torch

from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu


def none(*shape, dtype=torch.bfloat16):
    x = torch.tensor(np.zeros((0,) + shape, dtype=np.float32))       # strides of zeros
    assert set(x.stride()) == {0}
    return x.cuda().to(dtype)


def ints(*x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def test_append_and_attend():
    kv = tl.PagedKVCache(2, 16, 2, 64)
    q, k = none(4, 64), none(2, 64)
    norm = torch.ones(64, device="cuda")
    assert kv.append(k, k, ints(), ints(dtype=torch.int64), q=q).shape == (0, 4, 64)
    assert kv.append(k, k, ints(), ints(dtype=torch.int64), q=q, q_norm=norm, k_norm=norm).shape == (0, 4, 64)
    assert kv.attend(q, none(3, dtype=torch.int32), ints()).shape == (0, 4, 64)
    assert torch.count_nonzero(kv.k) == 0 and tl.tl_get_status() == tl.TL_OK


@pytest.mark.parametrize("requests", [0, 2])
def test_trees(requests):
    kv = tl.PagedKVCache(2, 16, 2, 64)
    starts, lens = ints(*[0] * (requests + 1)), ints(*[3] * requests)
    pages = torch.zeros((requests, 1), dtype=torch.int32, device="cuda") if requests else none(1, dtype=torch.int32)
    masks, positions, slots = kv.plan_tree(ints(), starts, lens, pages)
    assert kv.attend_tree(none(4, 64), masks, starts, pages, lens).shape == (0, 4, 64)
    for draft in (None, none(9, dtype=torch.float32)):
        path, counts, after = tl.tl_verify_tree(none(9, dtype=torch.float32), draft, ints(), ints(), starts, ints(dtype=torch.float32))
        assert path.shape == (0,) and counts.tolist() == [0] * requests and after.tolist() == [-1] * requests
    kv.compact(path, counts, starts, pages, lens)
    assert tl.tl_get_status() == tl.TL_OK
