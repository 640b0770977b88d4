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
