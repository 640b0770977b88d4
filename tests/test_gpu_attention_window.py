"""Windows beyond 32 bits: wider than any length is all of it, a negative one is refused whatever its low bits are."""

import pytest
import torch

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_paged_attention import build, check

pytestmark = pytest.mark.gpu


def test_windows_beyond_32_bits():
    lens = [40, 9]
    kv, q, table, k64, v64 = build(1, lens, 4, 2, 64, 16)
    good = check(kv, q, table, k64, v64, lens)
    args = q.cuda(), torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 62):
        assert torch.equal(kv.attend(*args, window=window), good)
    for window in (-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32, 5 - 2 ** 32, -2 ** 63):
        with pytest.raises(tl.TLError) as e:
            kv.attend(*args, window=window)
        assert e.value.code == tl.TL_EINVAL
    assert tl.tl_get_status() == tl.TL_OK
