"""The module that checks tensors for the serving operators refuses what is not a fitting CUDA tensor with a ValueError,
a wrong call with a TypeError, and never reaches the C ABI with it; no GPU."""

import pytest
import torch

from quantized_linear_layers_block_gb300 import build, tl


@pytest.fixture(scope="module")
def mod():
    build.build()
    return tl._tensors()


def test_number_of_arguments(mod):
    for f in (mod.kv_append, mod.paged_attention, mod.lora_apply):
        with pytest.raises(TypeError):
            f()
        with pytest.raises(TypeError):
            f(*[None] * 30)


def test_what_is_no_cuda_tensor(mod):
    x = torch.zeros(2, 2, 64)
    for bad in (x, None, 3, "k", [x]):
        with pytest.raises(ValueError):
            mod.kv_append(0, bad, x, None, x, None, False, None, None, None)
        with pytest.raises(ValueError):
            mod.paged_attention(0, bad, x, x, 1.0, 0, x, None, x, None)
        with pytest.raises(ValueError):
            mod.lora_apply(bad, x, x, x, 1, x, x, x, None)


def test_what_is_no_address(mod):
    with pytest.raises(TypeError):
        mod.kv_append("cache", None, None, None, None, None, False, None, None, None)
    with pytest.raises(OverflowError):
        mod.paged_attention(1 << 80, None, None, None, 1.0, 0, None, None, None, None)


def test_constructors_refuse_without_a_gpu():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for bad in (dict(dtype=torch.float32, k=k, v=k), dict(k=k), dict(k=k, v=k), dict(k=k, v=k, k_scale=torch.ones(2))):
        with pytest.raises(ValueError):
            tl.PagedKVCache(4, 16, 2, 64, **bad)
    A, B = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 32, 8, dtype=torch.bfloat16)
    for bad in ((A, B), (A.float(), B)):
        with pytest.raises(ValueError):
            tl.LoraBank(*bad)
    with pytest.raises(ValueError):
        tl.tl_lora_plan(torch.zeros(3, dtype=torch.int32), 2)
