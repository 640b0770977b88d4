"""GPU parity of tl_tree_attention against the 64-bit oracle (oracle/serving.py).

The tolerance is the rounding bound of the operator's arithmetic, for u = 2^-23 (a matrix instruction may truncate its fp32 sums):
  scores   E = (D / 16 + 21) u max_j scale sum |q k|   (D / 16 chained steps of 16 products)
  weights  2 (E + 2^-20) + split of p in two parts (2^-16)  relative, numerator and denominator
  sums     (n / 8 + 60) u    (two products of 16 keys a step, joins)
  output   half a unit in the last place of its type
"""

import numpy as np
import pytest
import torch

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_paged_attention import HALF_ULP, build

pytestmark = pytest.mark.gpu


def trees(rng, nodes, chain=False):
    """Parents of trees with so many nodes, and their masks."""
    parents = [[-1] + [i - 1 if chain else int(rng.integers(0, i)) for i in range(1, n)] if n else [] for n in nodes]
    return parents, [w for p in parents for w in O.tree_masks(p)]


def case(seed, lens, nodes, hq, hkv, d, page, cache="bf16", qtype=None, layout="heads", spread=1.0, pad=0, chain=False, masks=None):
    """(cache, q, masks, starts, table, k64, v64)"""
    total = [a + b for a, b in zip(lens, nodes)]
    kv, _, table, k64, v64 = build(seed, total, hq, hkv, d, page, cache, qtype, layout, spread)
    rng = np.random.default_rng(seed + 1)
    starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    words = masks if masks is not None else trees(rng, nodes, chain)[1]
    qt = torch.float16 if cache == "f16" or qtype == "f16" else torch.bfloat16
    q = torch.tensor(rng.standard_normal((int(starts[-1]) + pad, hq, d)).astype(np.float32)).to(qt)
    return kv, q, words + [0] * pad, starts, table, k64, v64


def attend(kv, q, words, starts, table, lens, **more):
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    kv.attend_tree(q.cuda(), torch.tensor(O.signed64(words)).cuda(), torch.tensor(starts).cuda(), torch.tensor(table).cuda(),
                   torch.tensor(lens, dtype=torch.int32).cuda(), out=out, lse=lse, **more)
    return out, lse


def compare(out, lse, q, words, starts, table, k64, v64, lens, window=0, sinks=0, scale=None):
    d = q.shape[2]
    used = int(starts[-1])
    assert torch.all(out[used:] == 9.0) and torch.all(lse[used:] == 7.0)          # padding is left as it was
    ref, ref_lse, (top, absv) = O.tree_attention(q[:used].double().numpy(), k64, v64, words, starts, table, lens, d ** -0.5 if scale is None else scale,
                                                 window, sinks)
    u = 2.0 ** -23
    E = (d / 16 + 21) * u * top + 2.0 ** -20
    n = max(lens) + 64
    tol = HALF_ULP[q.dtype] * np.abs(ref) + (2 * E[:, :, None] + 2.0 ** -16 + (n / 8 + 60) * u) * absv + 2.0 ** -24
    err = np.abs(out[:used].double().cpu().numpy() - ref)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(~(err <= tol))[:5].tolist())
    got = lse[:used].double().cpu().numpy()
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got - ref_lse)[~empty] <= (E + (n / 8 + 60) * u + 2.0 ** -22 * np.abs(ref_lse))[~empty])


def check(args, lens, window=0, sinks=0, scale=None, stream=None):
    kv, q, words, starts, table, k64, v64 = args
    out, lse = attend(kv, q, words, starts, table, lens, window=window, sinks=sinks, scale=scale, stream=stream)
    assert tl.tl_get_status(stream) == tl.TL_OK
    compare(out, lse, q, words, starts, table, k64, v64, lens, window, sinks, scale)
    return out


LENS = [0, 1, 15, 64, 63, 0, 65, 129, 300, 2]
NODES = [1, 3, 64, 7, 1, 0, 20, 33, 2, 64]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache,qtype", [("bf16", None), ("f16", None), ("f8", "bf16"), ("f8", "f16")])
def test_one_request(d, cache, qtype):
    check(case(d, [100], [5], 6, 2, d, 16, cache, qtype), [100])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache,qtype", [("bf16", None), ("f16", None), ("f8", "bf16"), ("f8", "f16")])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (12, 2), (5, 1), (33, 1)])
def test_types_and_head_sharing(d, cache, qtype, hq, hkv):
    check(case(d + hq, LENS, NODES, hq, hkv, d, 16, cache, qtype, pad=3), LENS)


@pytest.mark.parametrize("page", [1, 7, 16, 24, 100, 256])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_page_sizes_and_layouts(page, layout):
    for cache in ("bf16", "f8"):
        check(case(page, LENS, NODES, 6, 2, 128, page, cache, layout=layout), LENS)


@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 4), (65, 200), (100, 1), (128, 64), (200, 65), (1 << 20, 4), (1 << 40, 4)])
@pytest.mark.parametrize("d,cache", [(64, "f16"), (256, "bf16"), (128, "f8")])
def test_window_and_sinks(window, sinks, d, cache):
    lens = [0, 63, 64, 65, 130, 500, 1000]
    check(case(window % 1000 + sinks, lens, [2, 64, 3, 1, 30, 64, 10], 6, 2, d, 16, cache), lens, window, sinks)


def test_any_masks_and_rows_that_see_nothing():
    lens, nodes = [0, 0, 70, 5], [3, 64, 10, 40]
    rng = np.random.default_rng(7)
    words = [int(w) for w in rng.integers(0, 1 << 63, sum(nodes), dtype=np.uint64)]
    words[0], words[2], words[5], words[70] = 0, (1 << 64) - 8, 0, 0             # nothing; only bits that are no nodes; nothing; only cached ones
    for cache in ("bf16", "f8"):
        check(case(5, lens, nodes, 6, 2, 64, 16, cache, masks=list(words)), lens)


def test_long_requests_cut_over_many_blocks():
    for d, cache, lens in ((128, "bf16", [20000]), (64, "f8", [9000, 3]), (256, "f16", [5000, 6000])):
        check(case(d, lens, [4] * len(lens), 4, 2, d, 64, cache), lens)


def test_many_requests():
    rng = np.random.default_rng(3)
    lens, nodes = [int(x) for x in rng.integers(0, 90, 300)], [int(x) for x in rng.integers(0, 6, 300)]
    check(case(9, lens, nodes, 4, 2, 64, 16, pad=5), lens)


def test_large_scores_and_scales():
    # scores of some hundreds: the maximum grows and the sums are scaled down on the way; and a scale of zero, and a negative one
    for scale in (1.0, 0.0, -0.5):
        check(case(11, [400, 90], [9, 64], 6, 2, 64, 16, spread=3.0), [400, 90], scale=scale)
    check(case(12, [400, 90], [9, 64], 6, 2, 64, 16, "f16", spread=3.0), [400, 90], scale=1.0)


def test_query_strides_and_values_outside_f16():
    kv, q, words, starts, table, k64, v64 = case(13, [200], [12], 6, 2, 128, 16, "f8", "bf16")
    q = (q.float() * torch.tensor([1e30, 1.0, 1e-30, 1e-3, 70000.0, 1e3]).view(1, -1, 1)).to(torch.bfloat16)
    wide = torch.zeros((12, 9, 128), dtype=torch.bfloat16)
    wide[:, 2:8] = q
    dev = wide.cuda()[:, 2:8]
    args = [torch.tensor(O.signed64(words)).cuda(), torch.tensor(starts).cuda(), torch.tensor(table).cuda(), torch.tensor([200], dtype=torch.int32).cuda()]
    out, lse = torch.full_like(dev.contiguous(), 9.0), torch.full((12, 6), 7.0, device="cuda")
    kv.attend_tree(dev, *args, scale=1e-3, out=out, lse=lse)
    assert tl.tl_get_status() == tl.TL_OK
    ref, _, _ = O.tree_attention(q.double().numpy(), k64, v64, words, starts, table, [200], 1e-3)
    ok = [h for h in (1, 2, 3, 5)]               # the scores of the others are beyond any tolerance
    err = np.abs(out.double().cpu().numpy() - ref)[:, ok]
    assert np.all(err <= 2.0 ** -8 * np.abs(ref[:, ok]) + 2.0 ** -10)


@pytest.mark.parametrize("cache", ["bf16", "f16", "f8"])
@pytest.mark.parametrize("window", [0, 64])
def test_what_is_not_seen_has_no_influence(cache, window):
    """Values and keys that are infinite or NaN, in places that only some nodes see."""
    lens, nodes = [150, 30], [40, 10]
    args = case(17, lens, nodes, 4, 2, 64, 16, cache)
    kv, q, words, starts, table, k64, v64 = args
    clean, clean_lse = attend(kv, q, words, starts, table, lens, window=window, sinks=3 if window else 0)
    place = lens[0] + 6                             # node 6 of the first request; and the 61st cached place from the end
    early = lens[0] - 61
    for at, kinds in ((place, ("v", "k")), (early, ("v",))):
        page, row = int(table[0][at // 16]), at % 16
        sees = np.array([at in O.tree_seen(lens[0], words[t], window, 3 if window else 0) for t in range(40)] + [False] * 10)
        assert sees.any() and not sees.all()
        for kind in kinds:
            for value in ((float("nan"),) if cache == "f8" else (float("inf"), -float("inf"), float("nan"))):
                store = getattr(kv, kind)
                store = store.view(torch.uint8) if cache == "f8" else store
                kept = store[page, 1, row].clone()
                store[page, 1, row, 5] = 0x7F if cache == "f8" else value
                out, lse = attend(kv, q, words, starts, table, lens, window=window, sinks=3 if window else 0)
                store[page, 1, row] = kept
                assert torch.equal(out[:, :2], clean[:, :2])                   # the other key-value head
                assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], clean_lse[~sees])
                if kind == "v":
                    rest = [c for c in range(64) if c != 5]
                    assert torch.equal(out[:, :, rest], clean[:, :, rest])
                    hit = out[sees][:, 2:, 5]
                    assert torch.all(torch.isnan(hit)) if np.isnan(value) else torch.all(hit == value)
                elif np.isnan(value):
                    assert torch.all(torch.isnan(out[sees][:, 2:]))
    assert tl.tl_get_status() == tl.TL_OK


@pytest.mark.parametrize("cache", ["bf16", "f16"])
def test_infinite_values_that_all_see(cache):
    lens = [700]
    kv, q, words, starts, table, k64, v64 = case(19, lens, [12], 4, 2, 64, 16, cache, spread=4.0)
    for at in (5, 640):
        page, row = int(table[0][at // 16]), at % 16
        for c, value in ((3, float("inf")), (9, -float("inf"))):
            kept = kv.v[page, 0, row].clone()
            kv.v[page, 0, row, c] = value
            out, _ = attend(kv, q, words, starts, table, lens, scale=2.0)
            kv.v[page, 0, row] = kept
            assert torch.all(out[:, :2, c] == value)
            assert torch.isfinite(out[:, 2:]).all() and torch.isfinite(out[:, :2, [i for i in range(64) if i != c]]).all()


def test_a_chain_is_the_decode_steps():
    """Node i of a chain sees what attend() sees after i more tokens."""
    lens, n = [77, 300, 0], 6
    kv, q, words, starts, table, k64, v64 = case(21, lens, [n] * 3, 6, 2, 128, 16, chain=True)
    out, _ = attend(kv, q, words, starts, table, lens)
    for i in range(n):
        rows = [int(starts[b]) + i for b in range(3)]
        one = kv.attend(q[rows].cuda(), torch.tensor(table).cuda(), torch.tensor([x + i + 1 for x in lens], dtype=torch.int32).cuda())
        ref = one.double()
        assert torch.all((out[rows].double() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -14)      # both rounded to bf16


def test_same_result_on_every_run_and_in_a_graph():
    lens, nodes = [3000, 100, 0, 900], [9, 64, 2, 30]
    kv, q, words, starts, table, k64, v64 = case(23, lens, nodes, 12, 2, 128, 16, pad=2)
    dev = [q.cuda(), torch.tensor(O.signed64(words)).cuda(), torch.tensor(starts).cuda(), torch.tensor(table).cuda(),
           torch.tensor(lens, dtype=torch.int32).cuda()]
    first = kv.attend_tree(*dev)
    for _ in range(5):
        assert torch.equal(kv.attend_tree(*dev), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    with torch.cuda.stream(side):
        kv.attend_tree(*dev, out=out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kv.attend_tree(*dev, out=out)
    for new in (lens, [10, 0, 0, 500]):            # lengths are read on the device
        dev[4].copy_(torch.tensor(new, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kv.attend_tree(*dev))
    assert tl.tl_get_status() == tl.TL_OK


def test_two_streams_at_once():
    lens, nodes = [4000, 100], [9, 64]
    kv, q, words, starts, table, k64, v64 = case(25, lens, nodes, 12, 2, 64, 16)
    dev = [q.cuda(), torch.tensor(O.signed64(words)).cuda(), torch.tensor(starts).cuda(), torch.tensor(table).cuda(),
           torch.tensor(lens, dtype=torch.int32).cuda()]
    want = kv.attend_tree(*dev)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            got[i].append(kv.attend_tree(*dev, stream=st if i else st.cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for g in got for x in g)


def test_data_errors_are_reported():
    lens = [100, 40, 60]
    kv, q, words, starts, table, k64, v64 = case(27, lens, [5, 6, 7], 4, 2, 64, 16)
    good, _ = attend(kv, q, words, starts, table, lens)
    assert tl.tl_get_status() == tl.TL_OK

    def reported(keep, starts=starts, table=table, lens=lens):
        out, _ = attend(kv, q, words, starts, table, lens)
        assert tl.tl_get_status() == tl.TL_EDATA
        for b in keep:
            rows = slice(int(starts[b]), int(starts[b + 1]))
            assert torch.all((out[rows].double() - good[rows].double()).abs() <= 2.0 ** -7 * good[rows].double().abs() + 2.0 ** -14)

    for bad in (-1, 1 << 20):
        reported([0, 2], lens=[100, bad, 60])
        t = table.copy()
        t[1, 1] = bad
        reported([0, 2], table=t)
    reported([0, 2], lens=[100, table.shape[1] * 16 - 5, 60])                 # no room for its nodes
    for s in ([0, 5, 4, 4], [0, 5, 11, 99], [-3, 5, 11, 18]):
        keep = [b for b in range(3) if 0 <= s[b] <= s[b + 1] <= 18 and (s[b], s[b + 1]) == (starts[b], starts[b + 1])]
        reported(keep, starts=np.array(s, dtype=np.int32))
    kv2, q2, words2, starts2, table2, _, _ = case(28, [10], [64], 4, 2, 64, 16, pad=10)
    attend(kv2, q2, words2, np.array([0, 65], dtype=np.int32), table2, [10])
    assert tl.tl_get_status() == tl.TL_EDATA
