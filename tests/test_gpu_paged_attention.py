"""GPU parity of tl_paged_attention against the 64-bit oracle (oracle/serving.py).

The tolerance is the rounding bound of the operator's arithmetic, for u = 2^-23
(a matrix instruction may truncate its fp32 sums):
  scores   E = (D / 16 + 21) u max_j scale sum |q k|   (D / 16 chained steps of 16 products)
  weights  2 (E + 2^-20) + split of p in two parts (2^-16)  relative, numerator and denominator
  sums     (n / 16 + 40) u
  output   half a unit in the last place of its type
"""

import numpy as np
import pytest
import torch

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def build(seed, lens, hq, hkv, d, page, cache="bf16", qtype=None, layout="heads", spread=1.0, spare=2):
    """A cache with the requests' pages in random places; rows that no request owns hold NaN."""
    rng = np.random.default_rng(seed)
    dt = TYPES[cache]
    qt = TYPES[qtype or (cache if cache != "f8" else "bf16")]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(need + [1]) + 1), -7, dtype=np.int32)     # entries past the end are not read
    at = 0
    owned = np.zeros((pages, page), dtype=bool)
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for j in range(n):
            owned[table[b, j // page], j % page] = True
    ks = vs = None
    if cache == "f8":
        ks = torch.tensor(rng.uniform(0.01, 0.05, hkv).astype(np.float32))
        vs = torch.tensor(rng.uniform(0.01, 0.05, hkv).astype(np.float32))
    bufs = []
    for s in (ks, vs):
        x = torch.tensor(rng.standard_normal((pages, hkv, page, d)).astype(np.float32)) * spread
        if s is not None:
            x = (x / s.view(1, -1, 1, 1)).clamp(-448, 448)
        x[~torch.tensor(owned)[:, None, :].expand(pages, hkv, page)] = float("nan")
        x = x.to(dt)
        bufs.append(x)
    dev = []
    for x in bufs:
        if layout == "tokens":        # [pages, page_size, heads, dim] in memory
            dev.append(x.view(torch.uint8 if cache == "f8" else dt).transpose(1, 2).contiguous().cuda().view(dt).transpose(1, 2))
        else:
            dev.append(x.cuda())
    kv = tl.PagedKVCache(pages, page, hkv, d, dtype=dt, k=dev[0], v=dev[1],
                         k_scale=None if ks is None else ks.cuda(), v_scale=None if vs is None else vs.cuda())
    q = torch.tensor(rng.standard_normal((len(lens), hq, d)).astype(np.float32)).to(qt)
    k64, v64 = (np.nan_to_num(x.double().numpy()) * (1 if s is None else s.double().numpy()[None, :, None, None])
                for x, s in zip(bufs, (ks, vs)))
    return kv, q, table, k64, v64


def check(kv, q, table, k64, v64, lens, window=0, scale=None, out=None, stream=None):
    d = q.shape[2]
    sc = d ** -0.5 if scale is None else scale
    lse = torch.full((len(lens), q.shape[1]), 7.0, device="cuda")
    qd = q if q.is_cuda else q.cuda()
    y = kv.attend(qd, torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale, window=window,
                  out=out, lse=lse, stream=stream)
    assert tl.tl_get_status(stream) == tl.TL_OK
    ref, ref_lse, (top, absv) = O.paged_attention(q.double().cpu().numpy(), k64, v64, table, lens, sc, window)
    u = 2.0 ** -23
    E = (d / 16 + 21) * u * top + 2.0 ** -20
    n = max(lens) if len(lens) else 0
    tol = HALF_ULP[q.dtype] * np.abs(ref) + (2 * E[:, :, None] + 2.0 ** -16 + (n / 16 + 40) * u) * absv + 2.0 ** -24
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / tol).max())
    got = lse.double().cpu().numpy()
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got - ref_lse)[~empty] <= (E + (n / 16 + 40) * u + 2.0 ** -22 * np.abs(ref_lse))[~empty])
    assert np.all(y.double().cpu().numpy()[empty] == 0)
    return y


LENS = [0, 1, 15, 16, 17, 0, 63, 64, 65, 129, 300, 2]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache,qtype", [("bf16", None), ("f16", None), ("f8", "bf16"), ("f8", "f16")])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (24, 4), (10, 2), (8, 1), (12, 1), (16, 1), (17, 1), (33, 1)])
def test_types_and_head_sharing(d, cache, qtype, hq, hkv):
    args = build(d + hq, LENS, hq, hkv, d, 16, cache, qtype)
    check(*args, LENS)


@pytest.mark.parametrize("page", [1, 7, 16, 24, 100, 256])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_page_sizes_and_layouts(page, layout):
    for cache in ("bf16", "f8"):
        check(*build(page, LENS, 6, 2, 128, page, cache, layout=layout), LENS)


@pytest.mark.parametrize("window", [1, 5, 16, 64, 100, 1000])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 4), (256, 6, 1)])
def test_window(window, d, hq, hkv):
    check(*build(window, LENS, hq, hkv, d, 16), LENS, window=window)


@pytest.mark.parametrize("d,cache", [(64, "f16"), (128, "bf16"), (256, "bf16"), (128, "f8"), (256, "f8")])
@pytest.mark.parametrize("n", [1, 577, 5000])
def test_one_request_split_over_blocks(d, cache, n):
    args = build(n, [n], 6, 1, d, 16, cache)
    a = check(*args, [n])
    b = check(*args, [n])
    assert torch.equal(a, b)        # the order in which blocks arrive does not reach the result


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "f8"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 1), (12, 1), (20, 2), (33, 1)])
def test_few_short_requests(d, cache, hq, hkv):
    """Small calls, in which a cluster of blocks shares each segment."""
    for lens, window in (([1], 0), ([0, 70], 0), ([700, 64], 0), ([900], 100), ([33, 0], 1)):
        check(*build(d + hq + len(lens), lens, hq, hkv, d, 16, cache), lens, window=window)


@pytest.mark.parametrize("d,cache", [(64, "bf16"), (128, "f16"), (128, "f8"), (256, "bf16"), (256, "f8")])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 1), (40, 2)])
@pytest.mark.parametrize("batch,longest", [(2, 2040), (9, 1500), (14, 1000), (30, 700), (75, 460), (150, 250), (150, 30)])
def test_clusters_of_every_size(d, cache, hq, hkv, batch, longest):
    """From eight blocks to a segment down to one, with requests of no token and of one among them."""
    rng = np.random.default_rng(batch + d)
    lens = [longest, 0, 1] + [int(n) for n in rng.integers(2, longest, batch)]
    check(*build(batch + d + hq, lens[:batch], hq, hkv, d, 16, cache), lens[:batch])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache,qtype", [("bf16", None), ("f16", None), ("f8", "bf16"), ("f8", "f16")])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 1), (24, 2), (20, 1), (40, 1)])
def test_many_short_requests(d, cache, qtype, hq, hkv):
    """Segments of few keys, which a ring of a block takes whole: one for each ring, and several."""
    for b, hi, window in ((40, 95, 0), (700, 30, 0), (100, 110, 9), (3, 15, 0)):
        lens = [int(x) for x in np.random.default_rng(b + d).integers(0, hi + 1, b)]
        check(*build(d + hq + b, lens, hq, hkv, d, 16, cache, qtype), lens, window=window)


def test_bad_lengths_among_short_requests():
    lens = [5, 9, 3, 7] * 30
    kv, q, table, k64, v64 = build(22, lens, 4, 2, 64, 16)
    good = check(kv, q, table, k64, v64, lens)
    wrong = list(lens)
    wrong[50], wrong[51] = -3, 1000
    safe = np.where(table < 0, 0, table)
    y = kv.attend(q.cuda(), torch.tensor(safe).cuda(), torch.tensor(wrong, dtype=torch.int32).cuda())
    assert tl.tl_get_status() == tl.TL_EDATA
    keep = [i for i in range(120) if i not in (50, 51)]
    assert torch.equal(y[keep], good[keep])


def test_many_requests_and_workspace_reuse():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    kv, q, table, k64, v64 = build(5, lens, 4, 2, 64, 16)
    check(kv, q, table, k64, v64, lens)
    for part in (slice(0, 3), slice(100, 333), slice(0, 1)):      # other shapes through the same workspace
        check(kv, q[part], table[part], k64, v64, lens[part])


def test_ragged_long_batch():
    lens = [3000, 1, 0, 1200, 17, 2048, 5, 999]
    check(*build(11, lens, 10, 2, 128, 32), lens)


def test_scores_far_apart():
    """Scores of some hundreds: one key takes nearly all the weight and the running maximum moves often."""
    lens = [400, 33]
    check(*build(12, lens, 4, 1, 128, 16, spread=30.0), lens)
    check(*build(12, lens, 4, 1, 128, 16, "f16", spread=30.0), lens)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scale(scale):
    lens = [100, 1, 31]
    check(*build(13, lens, 4, 2, 64, 8), lens, scale=scale)


def test_bf16_query_with_an_8_bit_cache_keeps_its_range():
    """bf16 queries beyond f16's range, and tiny ones, over a cache that is widened to f16."""
    lens = [70, 20, 3]
    kv, q, table, k64, v64 = build(14, lens, 4, 2, 128, 16, "f8", "bf16")
    for mult in (2.0 ** 40, 2.0 ** -40):
        qm = (q.float() * mult).to(torch.bfloat16)
        check(kv, qm, table, k64, v64, lens, scale=128 ** -0.5 / mult)


def test_strided_query_and_output_on_another_stream():
    lens = [90, 200, 1]
    kv, q, table, k64, v64 = build(15, lens, 6, 2, 128, 16)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        wide = torch.full((3, 6 * 128 + 256), 3.0, dtype=torch.bfloat16, device="cuda")
        qs = wide[:, :6 * 128].view(3, 6, 128)
        qs.copy_(q.cuda())
        hold = torch.full((3, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        check(kv, qs, table, k64, v64, lens, out=hold[:, 1:7], stream=st)
        st.synchronize()
    assert bool((hold[:, 0] == 5).all()) and bool((hold[:, 7] == 5).all())


def test_another_stream_without_its_context():
    """The outputs and the workspace that a call allocates belong to the stream that it is given."""
    lens = [3000, 20]
    kv, q, table, k64, v64 = build(21, lens, 8, 2, 128, 16)
    qd, td, ld = q.cuda(), torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.empty((1 << 28,), dtype=torch.float32, device="cuda")
    for _ in range(20):
        busy.fill_(1.0)                  # the current stream is behind
    y = kv.attend(qd, td, ld, stream=st)
    st.synchronize()
    got = y.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, check(kv, q, table, k64, v64, lens))


def test_rows_past_the_32_bit_range():
    """A cache of over 2^31 elements, whose offsets in bytes pass 2^32, the request's pages at its end."""
    page, hkv, d = 64, 8, 128
    pages = 2 ** 31 // (page * hkv * d) + 40
    k = torch.empty((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    lens = [130, 64]
    table = np.array([[pages - 1, pages - 3, pages - 5], [pages - 2, -1, -1]], dtype=np.int32)
    g = torch.Generator().manual_seed(1)
    small_k = torch.randn((6, hkv, page, d), generator=g).to(torch.bfloat16)
    small_v = torch.randn((6, hkv, page, d), generator=g).to(torch.bfloat16)
    k[pages - 6:], v[pages - 6:] = small_k.cuda(), small_v.cuda()
    kv = tl.PagedKVCache(pages, page, hkv, d, k=k, v=v)
    q = torch.randn((2, 16, d), generator=g).to(torch.bfloat16)
    near = np.where(table >= 0, table - (pages - 6), -1)
    lse = torch.empty((2, 16), device="cuda")
    y = kv.attend(q.cuda(), torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), lse=lse)
    assert tl.tl_get_status() == tl.TL_OK
    ref, _, (top, absv) = O.paged_attention(q.double().numpy(), small_k.double().numpy(), small_v.double().numpy(), near, lens, d ** -0.5)
    tol = 2.0 ** -8 * np.abs(ref) + (2 * (29 * 2.0 ** -23 * top[:, :, None] + 2.0 ** -20) + 2.0 ** -15) * absv + 2.0 ** -24
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)


def test_bad_page_and_length_are_reported_and_leave_the_others_alone():
    lens = [100, 50, 80]
    kv, q, table, k64, v64 = build(16, lens, 4, 2, 64, 16)
    good = check(kv, q, table, k64, v64, lens)
    bad = table.copy()
    bad[1, 2] = kv.num_pages            # one past the end
    y = kv.attend(q.cuda(), torch.tensor(bad).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    assert tl.tl_get_status() == tl.TL_EDATA
    assert torch.equal(y[0], good[0]) and torch.equal(y[2], good[2])
    for wrong in (-1, table.shape[1] * 16 + 1):
        wl = [lens[0], wrong, lens[2]]
        t = table.copy()
        t[t < 0] = 0
        kv.attend(q.cuda(), torch.tensor(t).cuda(), torch.tensor(wl, dtype=torch.int32).cuda())
        assert tl.tl_get_status() == tl.TL_EDATA
    check(kv, q, table, k64, v64, lens)      # the workspace is clean again


def test_no_requests_and_no_pages():
    kv = tl.PagedKVCache(4, 16, 2, 64)
    y = kv.attend(torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 3), dtype=torch.int32, device="cuda"),
                  torch.empty((0,), dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 4, 64)
    y = kv.attend(torch.ones((2, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 0), dtype=torch.int32, device="cuda"),
                  torch.zeros((2,), dtype=torch.int32, device="cuda"))
    assert tl.tl_get_status() == tl.TL_OK and bool((y == 0).all())


def test_infinite_and_nan_keys_among_the_attended_ones():
    """What a request attends to does reach its result, and no other request's."""
    lens = [40, 40]
    kv, q, table, k64, v64 = build(17, lens, 2, 1, 64, 16)
    good = check(kv, q, table, k64, v64, lens)
    kv.k[table[0, 1], 0, 3] = float("nan")
    y = kv.attend(q.cuda(), torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    assert bool(torch.isnan(y[0]).all()) and torch.equal(y[1], good[1])


def test_graph_capture():
    lens = [300, 20]
    kv, q, table, k64, v64 = build(18, lens, 8, 2, 128, 16)
    good = check(kv, q, table, k64, v64, lens)
    qd, td, ld = q.cuda(), torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    out = torch.empty_like(qd)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            kv.attend(qd, td, ld, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, good)
    ld.copy_(torch.tensor([17, 20], dtype=torch.int32))     # lengths are read on the device
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1], kv.attend(qd, td, ld)[1]) and not torch.equal(out[0], good[0])


def test_binding_refusals():
    kv = tl.PagedKVCache(4, 16, 2, 64)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    pages = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    lens = torch.zeros((2,), dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(pages=pages.long()), dict(pages=pages[:1]),
                dict(lens=lens[:1]), dict(lens=lens.long()), dict(out=q[:1]), dict(lse=torch.zeros((2, 3), device="cuda"))):
        with pytest.raises(ValueError):
            kv.attend(**{**dict(q=q, pages=pages, lens=lens), **bad})
    with pytest.raises(tl.TLError):          # the cache's type and the query's differ
        kv.attend(q.half(), pages, lens)
    with pytest.raises(tl.TLError):          # 3 query heads on 2 key-value heads
        kv.attend(q[:, :3], pages, lens)
    with pytest.raises(tl.TLError):
        kv.attend(q, pages, lens, scale=float("inf"))
    with pytest.raises(tl.TLError):
        kv.attend(q, pages, lens, window=-1)
    with pytest.raises(tl.TLError) as e:
        tl.tl_paged_attention(kv, q, pages, lens, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == tl.TL_ENOSPACE
