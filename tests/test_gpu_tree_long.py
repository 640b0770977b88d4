"""Tree attention over long caches, where blocks go through many tiles, their rings many times round, and several row blocks share
the keys: a chain of nodes is as many requests of tl_paged_attention over the same pages.

Both results carry their type's half unit, and the bounds of the two kernels' arithmetic: scores of up to s = scale sum |q k| are off by
E = (D / 16 + 21) 2^-23 s, weights by 2 E + 2^-16, sums by (n / 8 + 60) 2^-23, all relative to sum p |v| / sum p. With normal
values, s < 4 sqrt(D) and weights peaked as here, that is below 2^-8 in all."""

import pytest
import torch

from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}


def filled(pages, page, hkv, d, cache, gen):
    scale = torch.full((hkv,), 0.02, device="cuda") if cache == "f8" else None
    kv = []
    for _ in range(2):
        x = torch.empty((pages, hkv, page, d), dtype=TYPES[cache], device="cuda")
        for i in range(0, pages, 256):
            y = torch.randn((min(256, pages - i), hkv, page, d), generator=gen, device="cuda")
            x[i:i + 256] = (y / 0.02 if cache == "f8" else y).to(x.dtype)
        kv.append(x)
    return tl.PagedKVCache(pages, page, hkv, d, dtype=TYPES[cache], k=kv[0], v=kv[1], k_scale=scale, v_scale=scale)


def chains(kv, lens, nodes, hq, gen, qtype, window=0):
    """Every request's tree is a chain of so many nodes. Returns tree attention's result and paged attention's."""
    B, page = len(lens), kv.page_size
    need = [-(-(n + nodes) // page) for n in lens]
    assert sum(need) <= kv.num_pages
    order = torch.randperm(kv.num_pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = torch.randn((B * nodes, hq, kv.head_dim), generator=gen, device="cuda").to(qtype)
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * nodes
    masks = torch.tensor([(1 << i + 1) - 1 if i < 63 else -1 for i in range(nodes)], device="cuda").repeat(B)
    scale = 4.0 * kv.head_dim ** -0.5
    got = kv.attend_tree(q, masks, starts, table, lens, scale=scale, window=window)
    one = kv.attend(q, table.repeat_interleave(nodes, 0), (lens.view(-1, 1) + torch.arange(1, nodes + 1, device="cuda")).int().view(-1), scale=scale, window=window)
    assert tl.tl_get_status() == tl.TL_OK
    return got.double(), one.double()


def same(got, one):
    err = (got - one).abs()
    tol = 2.0 ** -7 * one.abs() + 2.0 ** -8
    assert torch.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "f16", "f8"])
@pytest.mark.parametrize("page", [24, 64])
def test_many_tiles_to_a_block(d, cache, page):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    lens = [1500 + 331 * i for i in range(24)]
    kv = filled(24 * (11000 // page + 2), page, 4, d, cache, gen)
    qtype = torch.float16 if cache == "f16" else torch.bfloat16
    for nodes, hq in ((1, 8), (5, 20)):
        same(*chains(kv, lens, nodes, hq, gen, qtype))
    same(*chains(kv, lens, 2, 4, gen, qtype, window=1000))


@pytest.mark.parametrize("d,hkv,cache,n", [(256, 4, "bf16", 40000), (128, 2, "f16", 150000), (64, 4, "f8", 300000)])
def test_row_blocks_share_the_keys(d, hkv, cache, n):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    kv = filled(n // 64 + 60, 64, hkv, d, cache, gen)
    qtype = torch.float16 if cache == "f16" else torch.bfloat16
    same(*chains(kv, [n], 64, 6 * hkv, gen, qtype))
    same(*chains(kv, [n // 3, 700, n // 5], 33, 6 * hkv, gen, qtype))


def test_offsets_beyond_32_bits():
    """A cache whose last rows lie more than 2^32 bytes (and 2^31 elements) from its first."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    page, hkv, d = 64, 8, 128
    pages = (1 << 31) // (page * hkv * d) + 64
    k, v = (torch.zeros((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv = tl.PagedKVCache(pages, page, hkv, d, k=k, v=v)
    last = torch.arange(pages - 40, pages, dtype=torch.int32, device="cuda")
    for x in (k, v):
        x[-40:] = torch.randn((40, hkv, page, d), generator=gen, device="cuda").to(x.dtype)
    small = tl.PagedKVCache(40, page, hkv, d, k=k[-40:].clone(), v=v[-40:].clone())
    n, nodes = 2000, 6
    q = torch.randn((nodes, 16, d), generator=gen, device="cuda").to(torch.bfloat16)
    masks = torch.tensor([1, 3, 7, 9, 25, 33], device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    starts, lens = i32([0, nodes]), i32([n])
    a = kv.attend_tree(q, masks, starts, last[None], lens)
    b = small.attend_tree(q, masks, starts, last[None] - (pages - 40), lens)
    assert torch.equal(a, b)
    path, counts = i32([0, 2, 3, 5, -1, -1]), i32([4])
    kv.compact(path, counts, starts, last[None], lens)
    small.compact(path, counts, starts, last[None] - (pages - 40), lens)
    assert torch.equal(k[-40:], small.k) and torch.equal(v[-40:], small.v)
    slots = kv.plan_tree(i32([-1, 0, 1, 0, 3, 0]), starts, lens, last[None])[2]
    assert slots.tolist() == [(pages - 40 + (n + i) // page) * page + (n + i) % page for i in range(nodes)]
    assert tl.tl_get_status() == tl.TL_OK


def test_stream_handles_and_outputs_given():
    """Every call on a stream handle, with outputs given and not, is the call on the current stream."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    kv = filled(64, 16, 2, 64, "bf16", gen)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    parents, starts, lens = i32([-1, 0, 0, 1, -1, 0]), i32([0, 4, 6]), i32([70, 9])
    table = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    q = torch.randn((6, 4, 64), generator=gen, device="cuda").to(torch.bfloat16)
    kn, vn = (torch.randn((6, 2, 64), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand((64,), generator=gen, device="cuda") + 0.5
    target, draft = (torch.softmax(torch.randn((6, 300), generator=gen, device="cuda"), 1) for _ in range(2))
    tokens, uniform = i32([0, 5, 7, 9, 0, 11]), torch.rand((6,), generator=gen, device="cuda")

    def all_of(stream):
        masks, positions, slots = kv.plan_tree(parents, starts, lens, table, stream=stream)
        turned = kv.append(kn, vn, None, slots, q=q, q_norm=w, k_norm=w, stream=stream)
        out = kv.attend_tree(turned, masks, starts, table, lens, stream=stream)
        path, counts, after = tl.tl_verify_tree(target, draft, tokens, parents, starts, uniform, stream=stream)
        kv.compact(path, counts, starts, table, lens, stream=stream)
        return [masks, positions, slots, turned, out, path, counts, after, kv.k.clone() if stream is None else kv.k, kv.v.clone() if stream is None else kv.v]

    k, v = kv.k.clone(), kv.v.clone()
    want = all_of(None)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        kv.k.copy_(k)
        kv.v.copy_(v)
        torch.cuda.synchronize()
        got = all_of(stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tl.tl_get_status() == tl.TL_OK


def test_refusals():
    kv = tl.PagedKVCache(4, 16, 2, 64)
    odd = tl.PagedKVCache(4, 16, 2, 48)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    q, masks, starts, table, lens = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(3, dtype=torch.int64, device="cuda"), i32([0, 3]), \
        i32([[0, 1]]), i32([5])
    for more in (dict(window=-1), dict(sinks=4), dict(sinks=-1, window=100), dict(scale=float("nan"))):
        with pytest.raises(tl.TLError) as e:
            kv.attend_tree(q, masks, starts, table, lens, **more)
        assert e.value.code == tl.TL_EINVAL
    for cache, x, more in ((kv, q, dict(window=63)), (odd, torch.zeros((3, 4, 48), dtype=torch.bfloat16, device="cuda"), {})):
        with pytest.raises(tl.TLError) as e:
            cache.attend_tree(x, masks, starts, table, lens, **more)
        assert e.value.code == tl.TL_EUNSUPPORTED
    with pytest.raises(tl.TLError) as e:
        tl.tl_tree_attention(kv, q, masks, starts, table, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == tl.TL_ENOSPACE
    with pytest.raises(ValueError):
        kv.attend_tree(q.half(), masks, starts, table, lens, out=torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        kv.append(q[:, :2], q[:, 2:], None, torch.arange(3, device="cuda"), q_norm=torch.ones(63, device="cuda"), q=q)
    empty = kv.attend_tree(q[:0], masks[:0], i32([0, 0]), table, lens)
    assert empty.shape == (0, 4, 64)
    assert tl.tl_verify_tree(torch.rand(0, 7, device="cuda"), None, i32([]), i32([]), i32([0, 0]), torch.rand(0, device="cuda"))[1].tolist() == [0]
    assert tl.tl_get_status() == tl.TL_OK


def test_all_rows_are_padding():
    """No request, but rows: the outputs of padding."""
    kv = tl.PagedKVCache(4, 16, 2, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    none, pages = i32([]), torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    path, counts, after = tl.tl_verify_tree(torch.rand(5, 9, device="cuda"), None, i32([1] * 5), i32([-1] * 5), i32([0]), torch.rand(5, device="cuda"),
                                            path=i32([7] * 5))
    assert path.tolist() == [-1] * 5 and counts.numel() == after.numel() == 0
    masks, positions, slots = kv.plan_tree(i32([-1] * 5), i32([0]), none, pages)
    assert masks.tolist() == positions.tolist() == [0] * 5 and slots.tolist() == [-1] * 5
    out = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    kv.attend_tree(torch.ones_like(out), masks, i32([0]), pages, none, out=out)
    assert torch.all(out == 3.0)
    kv.compact(path, counts, i32([0]), pages, none)
    assert tl.tl_get_status() == tl.TL_OK


@pytest.mark.parametrize("hq,hkv,d,cache", [(128, 1, 64, "bf16"), (128, 1, 256, "f8"), (1024, 8, 128, "f16")])
def test_most_rows(hq, hkv, d, cache):
    """64 nodes of 128 heads on one: 64 row blocks to a request."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(hq + d)
    kv = filled(60, 16, hkv, d, cache, gen)
    qtype = torch.float16 if cache == "f16" else torch.bfloat16
    same(*chains(kv, [130, 0, 77], 64, hq, gen, qtype))


@pytest.mark.parametrize("cache,d,tiles", [("bf16", 256, 479), ("bf16", 256, 481), ("f16", 64, 470), ("f8", 128, 319), ("f8", 128, 322)])
def test_around_the_longest_clusters(cache, d, tiles):
    """One request on seven heads: sixteen blocks with up to 30 (8 bits: 20) tiles each, and the list beyond."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tiles)
    kv = filled(4 * (tiles + 1), 16, 7, d, cache, gen)
    qtype = torch.float16 if cache == "f16" else torch.bfloat16
    same(*chains(kv, [64 * tiles - 5], 5, 14, gen, qtype))
