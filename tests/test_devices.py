"""The serving operators' calls refuse tensors of different GPUs; no GPU (tensors without memory stand for those of two)."""

import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from quantized_linear_layers_block_gb300 import build, tl

# where torch finds a GPU it wants to reach each one that such a tensor names
pytestmark = pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2, reason="one GPU: tensors of another cannot be named")


@pytest.fixture(scope="module")
def mod():
    build.build()
    return tl._tensors()


def fake(gpu, shape, dtype):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=f"cuda:{gpu}")


BF, F, I, L, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
APPEND = [("k", (3, 2, 64), BF), ("v", (3, 2, 64), BF), ("positions", (3,), I), ("slots", (3,), L), ("cos_sin", (8, 64), F),
          ("interleaved", None, False), ("q", (3, 4, 64), BF), ("q_out", (3, 4, 64), BF), ("stream", None, None)]
ATTEND = [("q", (3, 4, 64), BF), ("pages", (3, 2), I), ("lens", (3,), I), ("scale", None, 1.0), ("window", None, 0), ("out", (3, 4, 64), BF),
          ("lse", (3, 4), F), ("workspace", (64,), U8), ("stream", None, None)]
ADAPT = [("A", (2, 8, 64), BF), ("B", (2, 32, 8), BF), ("scale", (2,), F), ("plan", (64,), U8), ("tokens", None, 3), ("x", (3, 64), BF),
         ("base", (3, 32), BF), ("out", (3, 32), BF), ("stream", None, None)]


def arguments(spec, away):
    """Tensors on GPU 0, the one named `away` on GPU 1."""
    return [x if shape is None else fake(int(name == away), shape, x) for name, shape, x in spec]


def tensors(spec):
    return [name for name, shape, _ in spec if shape is not None]


def refused(f, *args):
    with pytest.raises(ValueError, match="GPU"):
        f(*args)


@pytest.mark.parametrize("away", tensors(APPEND))
def test_append(mod, away):
    cache = tl._Cache(tl.tl_kv_cache(dtype=tl.TL_BF16, kv_heads=2, head_dim=64, page_size=16, num_pages=4), 0)
    refused(mod.kv_append, ctypes.addressof(cache), *arguments(APPEND, away))


@pytest.mark.parametrize("away", tensors(ATTEND))
def test_attend(mod, away):
    cache = tl._Cache(tl.tl_kv_cache(dtype=tl.TL_BF16, kv_heads=2, head_dim=64, page_size=16, num_pages=4), 0)
    refused(mod.paged_attention, ctypes.addressof(cache), *arguments(ATTEND, away))


@pytest.mark.parametrize("spec,f", [(APPEND, "kv_append"), (ATTEND, "paged_attention")])
def test_cache_on_another_gpu(mod, spec, f):
    cache = tl._Cache(tl.tl_kv_cache(dtype=tl.TL_BF16, kv_heads=2, head_dim=64, page_size=16, num_pages=4), 1)
    refused(getattr(mod, f), ctypes.addressof(cache), *arguments(spec, None))


@pytest.mark.parametrize("away", tensors(ADAPT))
def test_adapt(mod, away):
    refused(mod.lora_apply, *arguments(ADAPT, away))


def test_constructors():
    A, B, scale = fake(0, (2, 8, 64), BF), fake(0, (2, 32, 8), BF), fake(0, (2,), F)
    refused(tl.LoraBank, A, fake(1, (2, 32, 8), BF), scale)
    refused(tl.LoraBank, A, B, fake(1, (2,), F))
    k, v, s = fake(0, (4, 2, 16, 64), BF), fake(1, (4, 2, 16, 64), BF), fake(0, (2,), F)
    refused(lambda: tl.PagedKVCache(4, 16, 2, 64, k=k, v=v))
    f8 = torch.float8_e4m3fn
    refused(lambda: tl.PagedKVCache(4, 16, 2, 64, dtype=f8, k=fake(0, k.shape, f8), v=fake(0, k.shape, f8), k_scale=s, v_scale=fake(1, (2,), F)))
    refused(tl.tl_lora_plan, fake(0, (3,), I), 2, tl.LoraPlan(3, 2, fake(1, (64,), U8)))
