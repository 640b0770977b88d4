"""examples/decode_attention.py refuses the token that a request's pages do not hold, before anything is launched for it."""

import pytest
import torch

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_decode_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_full_request(example):  # noqa: F811
    h = example.AttentionHalf(2, 32, hidden=1024, q_heads=16, kv_heads=2, head_dim=64, rot_dim=64, adapters=2, rank=8)
    x = torch.ones((40, 1024), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        h.prompt(0, x[:33])
    h.prompt(0, x[:30])
    with pytest.raises(ValueError):
        h.prompt(0, x[:3])
    h.step(x[:2])
    h.step(x[:2])
    assert h.tokens == h.lens.tolist() == [32, 2]
    with pytest.raises(ValueError):
        h.step(x[:2])
    assert h.tokens == h.lens.tolist() == [32, 2] and tl.tl_get_status() == tl.TL_OK
