"""How many bits of A[a] x[m] count: B picks single elements of it, which are exact in fp32 here."""

import pytest
import torch

from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,bits", [(torch.float16, 22), (torch.bfloat16, 24)])
@pytest.mark.parametrize("rank", [8, 32, 128])
def test_bits_with_an_fp32_result(dtype, bits, rank):
    """h[m, r] = x[m, 0] A[r, 0] + x[m, 1] A[r, 1], all its digits below 24 bits: y[m, r] is h[m, r] up to the stated bits."""
    g = torch.Generator().manual_seed(rank)
    M, K = 40, 16
    x, A = torch.zeros(M, K), torch.zeros(1, rank, K)
    x[:, 0] = 1 + torch.randint(0, 128, (M,), generator=g) / 128               # 8 bits each, products of 16
    A[0, :, 0] = 1 + torch.randint(0, 128, (rank,), generator=g) / 128
    x[:, 1] = torch.randint(0, 16, (M,), generator=g) * 2.0 ** -11            # and 8 more below them: multiples of 2^-22
    A[0, :, 1] = torch.randint(0, 16, (rank,), generator=g) * 2.0 ** -11
    B = torch.eye(rank).view(1, rank, rank)
    h = x.double() @ A[0].double().t()
    assert torch.equal(h, h.float().double())
    x, A, B = (t.to(dtype).cuda() for t in (x, A, B))
    bank = tl.LoraBank(A, B)
    y = bank.apply(x, torch.zeros((M, rank), device="cuda"), bank.plan(torch.zeros(M, dtype=torch.int32, device="cuda")))
    assert tl.tl_get_status() == tl.TL_OK
    err = (y.double().cpu() - h).abs()
    assert bool((err <= 2.0 ** -bits * h.amax(1, keepdim=True)).all()), float(err.max())
