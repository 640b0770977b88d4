"""The attention half of a decoder layer, served for many requests at once.

Ternary projections (fused q, k and v; the output projection), each request's
low-rank adapters beside them, the paged key-value cache, and attention of one
new token per request, as a serving loop runs them:

    plan     = bank.plan(adapter of each request)          once per step, for every projection
    qkv      = adapters(x) + ternary(x)
    cache.append(k, v, positions, slots, q=q)              rotated on the way
    y        = cache.attend(q, pages, lens)
    out      = adapters(y) + ternary(y)

The step is captured in a CUDA graph: lengths, slots, pages and adapters are read
on the device, so one graph serves every step while the batch keeps its size.

    python examples/decode_attention.py [--requests 24] [--context 2000] [--steps 16] [--cache bf16|fp8]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_linear_layers_block_gb300 import tl  # noqa: E402


def random_ternary(n, k, gen, device):
    codes = torch.randint(-1, 2, (n, k), generator=gen, device=device, dtype=torch.int8)
    s = torch.exp(torch.randn((n, k // 128), generator=gen, device=device) * 0.4 - 4.0).to(torch.float16)
    return codes, s


class AttentionHalf:
    """One layer's projections, adapters and cache, with the buffers of a batch of `requests`."""

    def __init__(self, requests, max_context, hidden=5120, q_heads=24, kv_heads=4, head_dim=256, rot_dim=64, page_size=16, adapters=8,
                 rank=16, cache=torch.bfloat16, seed=0, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.shape = (q_heads, kv_heads, head_dim)
        width, inner = (q_heads + 2 * kv_heads) * head_dim, q_heads * head_dim
        self.weights = {"qkv": random_ternary(width, hidden, gen, device), "out": random_ternary(hidden, inner, gen, device)}
        self.qkv, self.out = (tl.TernaryLinear(*self.weights[n], device=device) for n in ("qkv", "out"))

        def bank(n, k):
            a = torch.randn((adapters, rank, k), generator=gen, device=device) / k ** 0.5
            b = torch.randn((adapters, n, rank), generator=gen, device=device) * 0.02
            return tl.LoraBank(a.to(torch.bfloat16), b.to(torch.bfloat16))

        self.qkv_bank, self.out_bank = bank(width, hidden), bank(hidden, inner)
        pages = requests * -(-max_context // page_size)
        scales = [None, None]
        if cache == torch.float8_e4m3fn:
            scales = [torch.full((kv_heads,), 0.05, device=device) for _ in range(2)]
        self.cache = tl.PagedKVCache(pages, page_size, kv_heads, head_dim, dtype=cache, k_scale=scales[0], v_scale=scales[1], device=device)
        half = rot_dim // 2
        rate = 10000.0 ** (-torch.arange(half, device=device, dtype=torch.float64) / half)
        angle = torch.arange(max_context, device=device, dtype=torch.float64)[:, None] * rate
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        # the scheduler's state: every request's pages (any order will do), length and adapter
        order = torch.randperm(pages, generator=gen, device=device, dtype=torch.int32)
        self.pages = order.view(requests, -1).contiguous()
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.max_context, self.tokens = max_context, [0] * requests        # (the lengths once more, on the host)
        self.adapter = torch.randint(-1, adapters, (requests,), generator=gen, device=device, dtype=torch.int32)
        self.plan = self.qkv_bank.plan(self.adapter)
        self.x = torch.empty((requests, hidden), dtype=torch.bfloat16, device=device)
        self.y = torch.empty((requests, hidden), dtype=torch.bfloat16, device=device)
        self.graph = None

    def slots(self, request, positions):
        """The slots of one request's tokens at `positions`."""
        size = self.cache.page_size
        p = positions.long()
        return self.pages[request, p // size].long() * size + p % size

    def project(self, x, plan):
        """x [T, hidden] -> q, k, v [T, heads, head_dim] as views of one tensor."""
        hq, hkv, d = self.shape
        qkv = self.qkv.forward(x)
        self.qkv_bank.apply(x, qkv, plan, out=qkv)
        q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
        return q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))

    def _take(self, requests, n):
        """n more tokens of each of these requests, whose pages have to hold them: their places are looked up unchecked."""
        full = [r for r in requests if self.tokens[r] + n > self.max_context]
        if full:
            raise ValueError(f"requests {full}: {n} more tokens are beyond {self.max_context}")
        for r in requests:
            self.tokens[r] += n

    def prompt(self, request, x):
        """Appends the keys and values of a prompt's tokens x [T, hidden] to one request."""
        begin = self.tokens[request]
        self._take([request], x.shape[0])
        at = torch.arange(begin, begin + x.shape[0], dtype=torch.int32, device=x.device)
        plan = self.qkv_bank.plan(self.adapter[request].expand(x.shape[0]).contiguous())
        _, k, v = self.project(x, plan)
        self.cache.append(k, v, at, self.slots(request, at), cos_sin=self.cos_sin)
        self.lens[request] += x.shape[0]

    def _step(self):
        requests = torch.arange(len(self.lens), device=self.lens.device)
        slots = self.slots(requests, self.lens)
        q, k, v = self.project(self.x, self.plan)
        self.cache.append(k, v, self.lens, slots, cos_sin=self.cos_sin, q=q, q_out=q)
        self.lens += 1
        attended = self.cache.attend(q, self.pages, self.lens).flatten(1)
        self.out.forward(attended, out=self.y)
        self.out_bank.apply(attended, self.y, self.plan, out=self.y)

    def step(self, x):
        """One new token of every request: x [requests, hidden] -> the half's output, in a buffer that the next step reuses."""
        self._take(range(len(self.tokens)), 1)
        self.x.copy_(x)
        if self.graph is None:                       # warm up and capture on a copy of the scheduler's state
            lens = self.lens.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self._step()
                self.lens.copy_(lens)
                side.synchronize()
                self.graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(self.graph, stream=side):
                    self._step()
            torch.cuda.current_stream().wait_stream(side)
        self.graph.replay()
        return self.y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=24)
    ap.add_argument("--context", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--cache", choices=["bf16", "fp8"], default="bf16")
    a = ap.parse_args(argv)
    half = AttentionHalf(a.requests, a.context + a.steps, cache=torch.float8_e4m3fn if a.cache == "fp8" else torch.bfloat16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for r in range(a.requests):
        n = max(1, a.context * (r + 1) // a.requests)
        half.prompt(r, torch.randn((n, half.qkv.K), generator=gen, device="cuda").to(torch.bfloat16))
    x = torch.randn((a.requests, half.qkv.K), generator=gen, device="cuda").to(torch.bfloat16)
    half.step(x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps - 1):
        x = half.step(x)
    end.record()
    torch.cuda.synchronize()
    if tl.tl_get_status() != tl.TL_OK:
        raise RuntimeError("a kernel reported an error")
    if a.steps > 1:
        us = begin.elapsed_time(end) * 1e3 / (a.steps - 1)
        print(f"{a.requests} requests of up to {a.context + a.steps} tokens: {us:.1f} us per step of the attention half")
    return half


if __name__ == "__main__":
    main()
