"""GPU tests of what a pass over drafted trees needs besides attention: plan, append with head norms, verification and
compaction, against plain forms (oracle/serving.py); and all of them together, as a server uses them."""

import numpy as np
import pytest
import torch

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_kv_append import angles

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def dev(x, dtype=None):
    return torch.as_tensor(np.asarray(x) if not isinstance(x, torch.Tensor) else x).to(dtype).cuda() if dtype else torch.as_tensor(np.asarray(x)).cuda()


def forest(rng, nodes, chain=False):
    return [[-1] + [i - 1 if chain else int(rng.integers(0, i)) for i in range(1, n)] if n else [] for n in nodes]


def table_for(rng, tokens, page, spare=2):
    need = [-(-n // page) for n in tokens]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(tokens), max(need + [1])), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


# ---------------------------------------------------------------- plan

@pytest.mark.parametrize("page", [1, 7, 16, 256])
@pytest.mark.parametrize("nodes", [[1], [64], [0], [0, 64, 1, 33, 0, 2, 32, 31, 63], list(range(1, 65)) * 8])
def test_plan(page, nodes):
    rng = np.random.default_rng(page + len(nodes))
    lens = [int(x) for x in rng.integers(0, 300, len(nodes))]
    table, pages = table_for(rng, [a + b for a, b in zip(lens, nodes)], page)
    parents = forest(rng, nodes)
    if len(nodes) > 1:
        parents[1][len(parents[1]) // 2] = -1                    # another root
    starts, pad = np.concatenate([[0], np.cumsum(nodes)]), 70
    kv = tl.PagedKVCache(pages, page, 1, 16)
    masks, positions, slots = kv.plan_tree(dev([x for p in parents for x in p] + [5] * pad, I32), dev(starts, I32), dev(lens, I32), dev(table))
    assert tl.tl_get_status() == tl.TL_OK
    words = [O.tree_masks(p) for p in parents]
    assert np.array_equal(masks.cpu().numpy(), O.signed64([w for ws in words for w in ws] + [0] * pad))
    assert positions.tolist() == [lens[b] + bin(w).count("1") - 1 for b, ws in enumerate(words) for w in ws] + [0] * pad
    at = [(b, lens[b] + i) for b, ws in enumerate(words) for i in range(len(ws))]
    assert slots.tolist() == [int(table[b][x // page]) * page + x % page for b, x in at] + [-1] * pad


def test_plan_chain_of_64():
    kv = tl.PagedKVCache(8, 16, 1, 16)
    masks, positions, _ = kv.plan_tree(dev([-1] + list(range(63)), I32), dev([0, 64], I32), dev([9], I32), dev([[0, 1, 2, 3, 4]], I32))
    assert masks.tolist() == [(1 << i + 1) - 1 if i < 63 else -1 for i in range(64)] and positions.tolist() == list(range(9, 73))


def test_plan_reports_data_errors():
    kv = tl.PagedKVCache(4, 16, 1, 16)
    good = dict(parents=[-1, 0, 1, -1, 0], starts=[0, 3, 5], lens=[4, 30], pages=[[0, 1], [2, 3]])

    def run(**change):
        a = {**good, **change}
        return kv.plan_tree(dev(a["parents"], I32), dev(a["starts"], I32), dev(a["lens"], I32), dev(a["pages"], I32))

    run()
    assert tl.tl_get_status() == tl.TL_OK
    for bad in (dict(parents=[-1, 0, 2, -1, 0]), dict(parents=[-2, 0, 1, -1, 0]), dict(starts=[0, 6, 5]), dict(starts=[0, 3, 6]), dict(starts=[-1, 3, 5]),
                dict(lens=[-1, 30]), dict(lens=[4, 31]), dict(lens=[2 ** 31 - 1, 30]), dict(pages=[[0, 1], [2, 4]]), dict(pages=[[-1, 1], [2, 3]])):
        masks, positions, slots = run(**bad)
        assert tl.tl_get_status() == tl.TL_EDATA, bad
        if "pages" in bad:
            assert -1 in slots.tolist()
    masks, _, _ = run(parents=[-1, 0, 2, -1, 0])                 # counts as a root
    assert tl.tl_get_status() == tl.TL_EDATA and masks.tolist() == [1, 3, 4, 1, 3]


# ---------------------------------------------------------------- append with norms

@pytest.mark.parametrize("d", [16, 48, 64, 80, 128, 256, 512])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f8"), ("f16", "f8")])
@pytest.mark.parametrize("T,norms", [(1, "qk"), (5, "q"), (200, "k"), (700, "qk")])
def test_append_norm(d, dtype, cache, T, norms):
    """Within half a unit of the stored type of the 64-bit formula, and the fp32 evaluation's own roundings: the sum of d squares
    in any order (d u / 2 of the norm), the mean, the root, two products and three of the rotation: (d / 2 + 8) u, u = 2^-24, of
    the two elements that a rotation mixes."""
    types = {"bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
    rng = np.random.default_rng(d + T)
    hq, hkv, page, rot, eps = 5, 3, 16, d // 32 * 16 if d > 16 else 16, 1e-5
    dt = types[dtype]
    rows = torch.tensor(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32) * 10.0 ** rng.uniform(-3, 2, (T, hq + 2 * hkv, 1)).astype(np.float32)).to(dt)
    rows[0, 0] = 0                                               # a head of zeros stays one
    wq, wk = (torch.tensor((1 + rng.standard_normal(d)).astype(np.float32)) for _ in range(2))
    cs, pos = angles(300, rot), rng.integers(0, 300, T).astype(np.int32)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    scale = torch.tensor(rng.uniform(0.01, 0.05, hkv).astype(np.float32)) if cache == "f8" else None
    kv = tl.PagedKVCache(pages, page, hkv, d, dtype=types[cache], k_scale=None if scale is None else scale.cuda(), v_scale=None if scale is None else scale.cuda())
    ref = tl.PagedKVCache(pages, page, hkv, d, dtype=types[cache], k_scale=None if scale is None else scale.cuda(), v_scale=None if scale is None else scale.cuda())
    r = rows.cuda()
    q, k, v = r[:, :hq], r[:, hq:hq + hkv], r[:, hq + hkv:]
    inter = bool(T % 2)
    got = kv.append(k, v, dev(pos), dev(slots), cos_sin=dev(cs), interleaved=inter, q=q, q_norm=wq.cuda() if "q" in norms else None,
                    k_norm=wk.cuda() if "k" in norms else None, eps=eps)
    assert tl.tl_get_status() == tl.TL_OK
    plain = ref.append(k, v, dev(pos), dev(slots), cos_sin=dev(cs), interleaved=inter, q=q)
    bytes_of = lambda t: t.contiguous().view(torch.uint8)        # noqa: E731
    assert torch.equal(bytes_of(kv.v), bytes_of(ref.v))          # values, and what has no norm, are append's
    if "q" not in norms:
        assert torch.equal(bytes_of(got), bytes_of(plain))
    if "k" not in norms:
        assert torch.equal(bytes_of(kv.k), bytes_of(ref.k))

    def formula(x, w):
        y = O.head_norm(x.double().numpy(), w.double().numpy(), eps)
        c, s = cs[pos][:, :rot // 2], cs[pos][:, rot // 2:]
        return O.rotate_rows(y, c, s, rot, inter), O.rotate_rows(np.abs(y), np.abs(c), -np.abs(s), rot, inter), \
            O.rotate_rows(np.abs(y), np.abs(c), np.abs(s), rot, inter)

    u = (d / 2 + 8) * 2.0 ** -24
    for name, x, w, have, s in (("q", rows[:, :hq], wq, got, None), ("k", rows[:, hq:hq + hkv], wk, kv.k, scale)):
        if name not in norms:
            continue
        want, big1, big2 = formula(x, w)
        big = np.maximum(np.abs(big1), np.abs(big2))
        if name == "k":
            have = have.view(torch.uint8)[dev(slots // page), :, dev(slots % page)].view(kv.dtype) if cache == "f8" else have[dev(slots // page), :, dev(slots % page)]
        have = have.double().cpu().numpy()
        if name == "k" and cache == "f8":
            s64 = s.double().numpy().reshape(1, -1, 1)
            want, big = np.clip(want / s64, -448, 448), big / s64
            half, least = 2.0 ** -4, 2.0 ** -10
        else:
            half, least = (2.0 ** -8, 1e-38) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25)
        tol = half * np.abs(want) + least + 2 * u * big
        assert np.all(np.abs(have - want) <= tol), float((np.abs(have - want) / tol).max())


def test_append_norm_in_place_padded_and_without_rotation():
    T, hq, hkv, d = 9, 4, 2, 64
    g = torch.Generator().manual_seed(0)
    rows = torch.randn((T, hq + 2 * hkv, d), generator=g).to(torch.bfloat16)
    w = 1 + torch.randn((d,), generator=g)
    kv = tl.PagedKVCache(2, 16, hkv, d)
    r = rows.cuda()
    slots = torch.arange(T)
    slots[4:] = -1
    q = kv.append(r[:, hq:hq + hkv], r[:, hq + hkv:], None, slots.cuda(), q=r[:, :hq], q_out=r[:, :hq], q_norm=w.cuda(), k_norm=w.cuda())
    assert tl.tl_get_status() == tl.TL_OK
    want = O.head_norm(rows[:, :hq].double().numpy(), w.double().numpy(), 1e-6)
    assert np.all(np.abs(q.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
    assert torch.count_nonzero(kv.k[0, :, 4:]) == 0 and torch.count_nonzero(kv.v[0, :, 4:]) == 0 and torch.count_nonzero(kv.k[0, :, :4]) > 0


# ---------------------------------------------------------------- verification

def draws(rng, nodes, vocab, drafted=True, chain=False, near=0.7):
    parents = forest(rng, nodes, chain)
    T = sum(nodes)

    def soft(x):
        e = np.exp(x - x.max(1, keepdims=True))
        return (e / e.sum(1, keepdims=True)).astype(np.float32)

    a, b = (rng.standard_normal((T, vocab)) * 2 for _ in range(2))
    target, draft = soft(a), soft(near * a + (1 - near ** 2) ** 0.5 * b)
    tokens = np.zeros(T, dtype=np.int32)
    row = 0
    for p in parents:
        for i, up in enumerate(p):
            if up >= 0:
                q = draft[row + up].astype(np.float64)
                tokens[row + i] = rng.choice(vocab, p=q / q.sum()) if drafted else rng.choice(np.argsort(target[row + up])[-3:])
        row += len(p)
    return parents, target, draft if drafted else None, tokens, rng.random(T).astype(np.float32)


def verified(parents, target, draft, tokens, uniform, nodes, pad=0, wide=0):
    T, vocab = target.shape

    def rows(x):
        full = torch.full((T + pad, vocab + wide), float("nan"))
        full[:T, :vocab] = torch.tensor(x)
        return full.cuda()[:, :vocab]

    z = np.zeros(pad)
    starts = np.concatenate([[0], np.cumsum(nodes)])
    got = tl.tl_verify_tree(rows(target), None if draft is None else rows(draft), dev(np.concatenate([tokens, z]), I32),
                            dev(np.concatenate([[x for p in parents for x in p], z]), I32), dev(starts, I32), dev(np.concatenate([uniform, z]), torch.float32))
    return [x.tolist() for x in got]


def expected(parents, target, draft, tokens, uniform, nodes, pad=0):
    path, counts, after, row = [], [], [], 0
    for p in parents:
        n = len(p)
        if n == 0:
            counts.append(0)
            after.append(-1)
            continue
        part = slice(row, row + n)
        way, x = O.verify_tree(target[part], None if draft is None else draft[part], tokens[part], p, uniform[part])
        path += way + [-1] * (n - len(way))
        counts.append(len(way))
        after.append(x)
        row += n
    return [path + [-1] * pad, counts, after]


@pytest.mark.parametrize("vocab", [1, 2, 3, 5, 128, 1000, 4099, 50001, 131072])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("chain", [True, False])
def test_verify(vocab, drafted, chain):
    rng = np.random.default_rng(vocab + drafted)
    nodes = [1, 8, 0, 5, 20] if vocab > 5000 else [1, 64, 0, 8, 30, 2, 17] * 5
    near = 0.7 if vocab > 2 else 0.2
    args = draws(rng, nodes, vocab, drafted, chain, near)
    for wide in (0, 1, 4):
        assert verified(*args, nodes, pad=3, wide=wide) == expected(*args, nodes, pad=3)
    assert tl.tl_get_status() == tl.TL_OK


@pytest.mark.parametrize("batch", [1, 2, 19, 40, 80, 160, 400])
def test_verify_batches(batch):
    rng = np.random.default_rng(batch)
    nodes = [int(x) for x in rng.integers(1, 12, batch)]
    args = draws(rng, nodes, 9000)
    assert verified(*args, nodes) == expected(*args, nodes)


def test_verify_edges():
    f = np.float32
    one = lambda i, n=6: np.eye(1, n, i, dtype=f)[0]             # noqa: E731
    even = np.full(6, 1 / 6, dtype=f)
    # the target is certain: only its token holds; the draft's own token with probability zero for the target never does
    t = np.stack([one(2), one(4), one(1)])
    assert verified([[-1, 0, 1]], t, None, np.array([0, 2, 4], dtype=np.int32), np.zeros(3, dtype=f), [3]) == [[0, 1, 2], [3], [1]]
    assert verified([[-1, 0, 1]], t, None, np.array([0, 2, 3], dtype=np.int32), np.zeros(3, dtype=f), [3]) == [[0, 1, -1], [2], [4]]
    # u = 0 accepts whatever the target can say; the largest u below one what the target says at least as often as the draft
    u = np.array([0, 1 - 2.0 ** -24], dtype=f)
    for p, want in ((even, [0, 1]), (np.array([.5, .1, .1, .1, .1, .1], dtype=f), [0, -1])):
        assert verified([[-1, 0]], np.stack([p, one(0)]), np.stack([even, even]), np.array([0, 1], dtype=np.int32), u, [2])[0] == want
    # nothing is left where the draft covers the target: the target's own row
    assert verified([[-1, 0]], np.stack([one(3), one(0)]), np.stack([one(3), one(3)]), np.array([0, 5], dtype=np.int32), np.full(2, .5, dtype=f), [2]) == \
        [[0, -1], [1], [3]]
    # a row of zeros ends at the last token; the same token twice among siblings; numbers outside [0, 1)
    assert verified([[-1]], np.zeros((1, 6), dtype=f), None, np.zeros(1, dtype=np.int32), np.full(1, .5, dtype=f), [1])[2] == [5]
    twice = [[-1, 0, 0]], np.stack([even] * 3), None, np.array([0, 3, 3], dtype=np.int32), np.array([.99, .9, .0], dtype=f), [3]
    assert verified(*twice) == [[0, -1, -1], [1], [5]]
    for x, want in ((-1.0, 0), (0.0, 0), (1.0, 5), (2.0, 5), (float("nan"), 0), (float("inf"), 5)):
        assert verified([[-1]], even[None], None, np.zeros(1, dtype=np.int32), np.array([x], dtype=f), [1])[2] == [want]
    # NaN and negative probabilities count as none, whatever else is in the row
    odd = np.array([float("nan"), -1, .25, float("-inf"), .25, .5], dtype=f)
    for x, want in ((0.0, 2), (0.24, 2), (0.26, 4), (0.6, 5)):
        assert verified([[-1]], odd[None], None, np.zeros(1, dtype=np.int32), np.array([x], dtype=f), [1])[2] == [want]
    assert tl.tl_get_status() == tl.TL_OK
    big = np.full((1, 20000), 3e38, dtype=f)                     # no distribution: some token, within the vocabulary
    assert 0 <= verified([[-1]], big, None, np.zeros(1, dtype=np.int32), np.array([.7], dtype=f), [1])[2][0] < 20000


def test_verify_emits_the_targets_distribution():
    """What two drafted siblings and a token after them emit first is distributed as the target, to 5 standard deviations."""
    rng = np.random.default_rng(5)
    n, vocab = 40000, 8
    p, q = rng.dirichlet(np.ones(vocab)).astype(np.float32), rng.dirichlet(np.ones(vocab)).astype(np.float32)
    nodes = [3] * n
    q64 = q.astype(np.float64) / q.astype(np.float64).sum()
    tokens = np.zeros((n, 3), dtype=np.int32)
    tokens[:, 1:] = rng.choice(vocab, (n, 2), p=q64)
    target, draft = (np.broadcast_to(x, (3 * n, vocab)) for x in (p, q))
    path, counts, after = verified([[-1, 0, 0]] * n, target, draft, tokens.reshape(-1), rng.random(3 * n).astype(np.float32), nodes)
    path = np.array(path).reshape(n, 3)
    first = np.where(np.array(counts) > 1, tokens[np.arange(n), np.maximum(path[:, 1], 0)], after)
    share = np.bincount(first, minlength=vocab) / n
    assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / n) + 1e-6)


def test_verify_reports_data_errors():
    rng = np.random.default_rng(1)
    nodes = [3, 4]
    parents, target, draft, tokens, uniform = draws(rng, nodes, 100)
    want = expected(parents, target, draft, tokens, uniform, nodes)
    bad = tokens.copy()
    bad[1] = 100
    got = verified(parents, target, draft, bad, uniform, nodes)
    assert tl.tl_get_status() == tl.TL_EDATA and got[0][3:] == want[0][3:] and got[1][1] == want[1][1] and got[2][1] == want[2][1]
    for p in ([[-1, 1, 0], parents[1]], [[-1, -2, 0], parents[1]]):
        got = verified(p, target, draft, tokens, uniform, nodes)
        assert tl.tl_get_status() == tl.TL_EDATA and got[1][1] == want[1][1]
    t = dev(target)
    for s in ([0, 8, 7], [0, 3, 8], [-1, 3, 7]):
        tl.tl_verify_tree(t, None, dev(tokens, I32), dev([x for p in parents for x in p], I32), dev(s, I32), dev(uniform))
        assert tl.tl_get_status() == tl.TL_EDATA


# ---------------------------------------------------------------- compaction

@pytest.mark.parametrize("cache", ["bf16", "f16", "f8"])
@pytest.mark.parametrize("page,d,hkv", [(16, 64, 2), (1, 16, 1), (7, 48, 3), (64, 256, 4), (256, 512, 1)])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_compact(cache, page, d, hkv, layout):
    rng = np.random.default_rng(page)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}[cache]
    nodes = [64, 1, 0, 64, 10, 5, 64]
    lens = [0, 3, 9, 100, 17, 250, 31]
    counts = [64, 1, 0, 40, 5, 0, 2]
    path = []
    for i, (n, c) in enumerate(zip(nodes, counts)):
        way = sorted(rng.choice(np.arange(1, n), c - 1, replace=False).tolist()) if c else []
        path += ([0] + way if c else []) + [-1] * (n - c)
    path[-64:-62] = [3, 60]                                      # node 0 itself is not on it: any increasing nodes move
    table, pages = table_for(rng, [a + b for a, b in zip(lens, nodes)], page)
    data = [rng.integers(0, 200, (pages, hkv, page, d * (1 if cache == "f8" else 2)), dtype=np.uint8) & 0x3F for _ in range(2)]
    bufs = []
    for x in data:
        t = torch.tensor(x)
        if layout == "tokens":
            bufs.append(t.transpose(1, 2).contiguous().cuda().view(dt).transpose(1, 2))
        else:
            bufs.append(t.cuda().view(dt))
    scale = torch.ones(hkv, device="cuda") if cache == "f8" else None
    kv = tl.PagedKVCache(pages, page, hkv, d, dtype=dt, k=bufs[0], v=bufs[1], k_scale=scale, v_scale=scale)
    starts = np.concatenate([[0], np.cumsum(nodes)])
    kv.compact(dev(path, I32), dev(counts, I32), dev(starts, I32), dev(table), dev(lens, I32))
    assert tl.tl_get_status() == tl.TL_OK
    for x, have in zip(data, (kv.k, kv.v)):
        want = x.copy()
        for b, n in enumerate(lens):
            moves = [(n + path[starts[b] + j], n + j) for j in range(counts[b])]
            rows = [x[table[b][a // page], :, a % page].copy() for a, _ in moves]
            for row, (_, z) in zip(rows, moves):
                want[table[b][z // page], :, z % page] = row
        got = have.transpose(1, 2).contiguous().view(torch.uint8).transpose(1, 2) if layout == "tokens" else have.view(torch.uint8)
        assert np.array_equal(got.cpu().numpy(), want)


def test_compact_reports_data_errors_and_leaves_the_request():
    kv = tl.PagedKVCache(8, 16, 2, 64)
    kv.k.normal_()
    kv.v.normal_()
    good = dict(path=[0, 2, 3, -1, 0, 3, -1, -1], counts=[3, 2], starts=[0, 4, 8], pages=[[0, 1], [2, 3]], lens=[5, 20])
    for bad in (dict(path=[0, 3, 2, -1, 0, 3, -1, -1]), dict(path=[0, 2, 4, -1, 0, 3, -1, -1]), dict(path=[-1, 2, 3, -1, 0, 3, -1, -1]),
                dict(path=[0, 2, 2, -1, 0, 3, -1, -1]), dict(counts=[5, 2]), dict(counts=[-1, 2]), dict(starts=[-1, 4, 8]), dict(lens=[-1, 20]),
                dict(lens=[29, 20]), dict(pages=[[9, 1], [2, 3]]), dict(pages=[[-1, 1], [2, 3]])):
        a = {**good, **bad}
        k, v = kv.k.clone(), kv.v.clone()
        kv.compact(dev(a["path"], I32), dev(a["counts"], I32), dev(a["starts"], I32), dev(a["pages"], I32), dev(a["lens"], I32))
        assert tl.tl_get_status() == tl.TL_EDATA, bad
        k[3, :, 5], v[3, :, 5] = k[3, :, 7], v[3, :, 7]          # the other request's rows have moved: place 20 + 3 to 20 + 1
        assert torch.equal(kv.k, k) and torch.equal(kv.v, v), bad


# ---------------------------------------------------------------- together

def test_a_round_of_drafting():
    """Plan, append, attend, verify and compact as a server runs them, twice, in a CUDA graph: afterwards the cache holds what
    appending the accepted tokens one by one would have put there, and attention over it agrees."""
    rng = np.random.default_rng(3)
    hq, hkv, d, page, vocab, B, n = 6, 2, 64, 16, 500, 5, 7
    lens0 = [0, 5, 33, 100, 60]
    table, pages = table_for(rng, [x + 40 for x in lens0], page)
    kv, ref = tl.PagedKVCache(pages, page, hkv, d), tl.PagedKVCache(pages, page, hkv, d)
    for a, b in ((kv.k, ref.k), (kv.v, ref.v)):
        a.copy_(torch.tensor(rng.standard_normal(a.shape).astype(np.float32)))
        b.copy_(a)
    cs = dev(angles(300, d))
    wq, wk = (dev((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)) for _ in range(2))
    T, pad = B * n, 3
    starts = np.arange(B + 1) * n
    buf = dict(parents=torch.zeros(T + pad, dtype=I32), tokens=torch.zeros(T + pad, dtype=I32), uniform=torch.zeros(T + pad), lens=torch.tensor(lens0, dtype=I32),
               qkv=torch.zeros((T + pad, hq + 2 * hkv, d), dtype=torch.bfloat16), target=torch.zeros((T + pad, vocab)), draft=torch.zeros((T + pad, vocab)))
    buf = {k: x.cuda() for k, x in buf.items()}
    st, tb = dev(starts, I32), dev(table)
    got = {}

    def step():
        masks, positions, slots = kv.plan_tree(buf["parents"], st, buf["lens"], tb)
        q, k, v = buf["qkv"].split([hq, hkv, hkv], dim=1)
        q = kv.append(k, v, positions, slots, cos_sin=cs, q=q, q_norm=wq, k_norm=wk)
        got["q"], got["out"] = q, kv.attend_tree(q, masks, st, tb, buf["lens"])
        got["path"], got["counts"], got["next"] = tl.tl_verify_tree(buf["target"], buf["draft"], buf["tokens"], buf["parents"], st, buf["uniform"])
        kv.compact(got["path"], got["counts"], st, tb, buf["lens"])
        buf["lens"].add_(got["counts"])

    graph, lens = None, list(lens0)
    for turn in range(3):
        nodes = [n] * B
        parents, target, draft, tokens, uniform = draws(rng, nodes, vocab, near=0.95)
        flat = [x for p in parents for x in p]
        for key, x in (("parents", flat), ("tokens", tokens), ("uniform", uniform), ("target", target), ("draft", draft)):
            buf[key][:T].copy_(torch.as_tensor(np.asarray(x)))
        rows = torch.tensor(rng.standard_normal((T + pad, hq + 2 * hkv, d)).astype(np.float32)).to(torch.bfloat16)
        buf["qkv"].copy_(rows)
        if graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
                side.synchronize()
                for a, b in ((kv.k, ref.k), (kv.v, ref.v)):
                    a.copy_(b)
                buf["lens"].copy_(torch.tensor(lens, dtype=I32))
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
            torch.cuda.current_stream().wait_stream(side)
        graph.replay()
        torch.cuda.synchronize()
        assert tl.tl_get_status() == tl.TL_OK
        want = expected(parents, target, draft, tokens, uniform, nodes, pad=pad)
        assert [got[k].tolist() for k in ("path", "counts", "next")] == want
        # the accepted tokens one by one, in the other cache
        for b in range(B):
            for j in range(want[1][b]):
                t = b * n + want[0][b * n + j]
                r = rows[t:t + 1].cuda()
                at = lens[b] + j
                slot = dev([int(table[b][at // page]) * page + at % page], I64)
                q1 = ref.append(r[:, hq:hq + hkv], r[:, hq + hkv:], dev([at], I32), slot, cos_sin=cs, q=r[:, :hq], q_norm=wq, k_norm=wk)
                assert torch.equal(q1[0], got["q"][t])
                one = ref.attend(q1, tb[b:b + 1], dev([at + 1], I32)).double()
                assert torch.all((got["out"][t].double() - one[0]).abs() <= 2.0 ** -7 * one[0].abs() + 2.0 ** -13)
            lens[b] += want[1][b]
            at = np.arange(lens[b])
            where = dev(table[b][at // page].astype(np.int64)), dev(at % page)
            for a, c in ((kv.k, ref.k), (kv.v, ref.v)):
                assert torch.equal(a[where[0], :, where[1]], c[where[0], :, where[1]])
        assert buf["lens"].tolist() == lens
