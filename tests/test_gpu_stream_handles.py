"""The serving operators on a stream that is given by its handle, and objects made on another stream than the one that uses
them first."""

import numpy as np
import pytest
import torch

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_lora import check as lora_check, make
from tests.test_gpu_paged_attention import build, check

pytestmark = pytest.mark.gpu


def keep_current_stream_behind():
    busy = torch.empty((1 << 28,), dtype=torch.float32, device="cuda")
    for _ in range(20):
        busy.fill_(1.0)


def test_results_of_a_call_on_a_handle_are_that_streams_memory():
    """A tensor of the result's size is freed while the current stream has yet to write it: it is not the result."""
    lens = [300, 20]
    kv, q, table, k64, v64 = build(21, lens, 8, 2, 128, 16)
    qd, td, ld = q.cuda(), torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    x, A, B, scale, base, ids = (t.cuda() if torch.is_tensor(t) else t for t in make(9, 45, 264, 200, 16, 3))
    ids = torch.tensor(ids).cuda()
    bank = tl.LoraBank(A, B, scale)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep_current_stream_behind()
    for like in (qd, base, torch.empty(tl.tl_lora_plan_size(45, 3), dtype=torch.uint8, device="cuda")):
        torch.empty_like(like).fill_(3)
    y = kv.attend(qd, td, ld, stream=st.cuda_stream)
    plan = bank.plan(ids, stream=st.cuda_stream)
    z = bank.apply(x, base, plan, stream=st.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, check(kv, q, table, k64, v64, lens))
    assert torch.equal(z, lora_check(*(t.cpu() for t in (x, A, B, scale, base)), ids.cpu().numpy()))


@pytest.mark.parametrize("handle", [0, None])
def test_default_stream(handle):
    lens = [70, 3]
    kv, q, table, k64, v64 = build(22, lens, 4, 2, 64, 16)
    qd, td, ld = q.cuda(), torch.tensor(table).cuda(), torch.tensor(np.asarray(lens, dtype=np.int32)).cuda()
    assert torch.equal(kv.attend(qd, td, ld, stream=handle), check(kv, q, table, k64, v64, lens))


def test_objects_made_on_a_stream_that_is_behind():
    """A cache's workspace (and its own k and v) and a bank's scales are there when the constructor returns, on any stream."""
    lens = [3000, 20]
    kv, q, table, k64, v64 = build(21, lens, 8, 2, 128, 16)
    qd, td, ld = q.cuda(), torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    good = check(kv, q, table, k64, v64, lens)
    x, A, B, scale, base, ids = (t.cuda() if torch.is_tensor(t) else t for t in make(9, 45, 264, 200, 16, 3))
    ids = torch.tensor(ids).cuda()
    ones = tl.LoraBank(A, B, torch.ones_like(scale))
    expected = ones.apply(x, base, ones.plan(ids))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    dirty = [torch.full_like(kv._ws, 7), torch.full_like(scale, 9.0)]      # where the new ones may lie
    keep_current_stream_behind()
    del dirty
    again = tl.PagedKVCache(kv.num_pages, kv.page_size, kv.kv_heads, kv.head_dim, k=kv.k, v=kv.v)
    keep_current_stream_behind()
    empty = tl.PagedKVCache(kv.num_pages, kv.page_size, kv.kv_heads, kv.head_dim)
    keep_current_stream_behind()
    bank = tl.LoraBank(A, B)
    y = again.attend(qd, td, ld, stream=st)
    z = bank.apply(x, base, bank.plan(ids, stream=st), stream=st)
    zero = empty.attend(qd, td.clamp(min=0), ld, stream=st)
    st.synchronize()
    assert torch.equal(y, good) and torch.equal(z, expected) and not zero.any()
