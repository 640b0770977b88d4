"""examples/decode_attention.py against the 64-bit oracle, step by step: the cache's contents, and the attention half's
output from the same cache. Projections in between are the layer's own (tested elsewhere), taken from the example."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_attention", os.path.join(ROOT, "examples", "decode_attention.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_steps_match_the_oracle(example, cache):
    h = example.AttentionHalf(3, 64, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, rot_dim=64, adapters=2, rank=8, cache=cache)
    hq, hkv, d = h.shape
    g = torch.Generator(device="cuda").manual_seed(3)
    seen = [[] for _ in range(3)]          # every request's inputs, in order
    for r, n in enumerate((1, 17, 40)):
        x = torch.randn((n, 1024), generator=g, device="cuda").to(torch.bfloat16)
        h.prompt(r, x)
        seen[r].append(x)
    cs = h.cos_sin.cpu().numpy()
    for _ in range(4):
        x = torch.randn((3, 1024), generator=g, device="cuda").to(torch.bfloat16)
        y = h.step(x).clone()
        torch.cuda.synchronize()
        assert tl.tl_get_status() == tl.TL_OK
        for r in range(3):
            seen[r].append(x[r:r + 1])
        lens = h.lens.tolist()
        assert lens == [sum(len(t) for t in s) for s in seen]
        # the cache, as the last token of each request should stand in it: the oracle's rotation of the projections
        q, k, v = (t.float().cpu().numpy() for t in h.project(x, h.plan))
        at = np.array(lens) - 1
        k = O.rotate_rows(k, cs[at, :32], cs[at, 32:], 64, False, np.float32)
        q = torch.tensor(O.rotate_rows(q, cs[at, :32], cs[at, 32:], 64, False, np.float32)).to(torch.bfloat16)
        pages = h.pages.cpu().numpy()
        stored = []
        for rows, scale, buf in ((k, h.cache.k_scale, h.cache.k), (v, h.cache.v_scale, h.cache.v)):
            rows = torch.tensor(rows)
            if scale is not None:
                rows = (rows * (1.0 / scale.cpu()).view(1, -1, 1)).clamp(-448, 448)
            got = torch.stack([buf[pages[r, at[r] // 16], :, at[r] % 16] for r in range(3)])
            assert torch.equal(got.float().cpu(), rows.to(cache).float())
            f = buf.float().double().cpu().numpy()
            stored.append(f if scale is None else f * scale.double().cpu().numpy()[None, :, None, None])
        # attention over what the cache holds, then the output projection and its adapter of the rounded result
        ref, _, _ = O.paged_attention(q.double().numpy(), stored[0], stored[1], pages, lens, d ** -0.5)
        attended = h.cache.attend(q.cuda(), h.pages, h.lens)
        # within half a unit in the last place of bf16 of the 64-bit result; the bound of the sums is far below it here
        err = np.abs(attended.double().cpu().numpy() - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * np.abs(stored[1]).max())
        out = h.out.forward(attended.flatten(1))
        again = h.out_bank.apply(attended.flatten(1), out, h.plan)
        assert torch.equal(y, again)


def test_command_runs(example, capsys):
    example.main(["--requests", "5", "--context", "70", "--steps", "3", "--cache", "fp8"])
    assert "5 requests" in capsys.readouterr().out
