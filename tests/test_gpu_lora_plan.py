"""A plan that is not of the call's batch is refused on the device before more of it is read than any plan has: here it ends
where its own items end, so nothing past it is this test's to read."""

import numpy as np
import pytest
import torch

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_lora import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,n,other_M,other_n", [(40, 3, 1, 3), (3000, 3, 2, 3), (1024, 5, 1023, 5), (40, 200, 40, 1), (1, 1, 40, 3), (40, 3, 3000, 64)])
@pytest.mark.parametrize("rank", [16, 64])
def test_plan_of_another_batch(M, n, other_M, other_n, rank):
    x, A, B, scale, base, ids = make(M + other_M + rank, M, 520, 264, rank, n)
    bank = tl.LoraBank(A.cuda(), B.cuda(), scale.cuda())
    other = tl.tl_lora_plan(torch.zeros(other_M, dtype=torch.int32, device="cuda"), other_n)
    hold = torch.full((M, 264), 7.0, dtype=base.dtype, device="cuda")
    bank.apply(x.cuda(), base.cuda(), tl.LoraPlan(M, n, other.data), out=hold)
    assert tl.tl_get_status() == tl.TL_EDATA and bool((hold == 7).all())
    check(x, A, B, scale, base, ids)


@pytest.mark.parametrize("M,n", [(1, 1), (1, 64), (48, 256), (300, 100), (2000, 64)])
@pytest.mark.parametrize("rank", [16, 64])
def test_fewer_items_than_the_grid_has_places_for(M, n, rank):
    """All tokens of one adapter of many, and of none: most blocks find no item."""
    for a in (n - 1, 0, -1):
        check(*make(M + n + rank, M, 520, 264, rank, n, ids=np.full(M, a)))
