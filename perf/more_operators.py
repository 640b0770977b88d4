"""What is measured of the operators by which a server drafts several tokens ahead and checks them in one pass of its model.

A request's drafted tokens form a tree: node 0 is the last token that is already
certain, every other node one guess at what follows its parent. One pass of the
model takes all nodes of all requests, ragged, behind each other:

  plan     the tree's ancestor masks, positions and cache slots, from its parents
  append   the nodes' keys and values go into the paged cache; queries and keys
           are normalised for each head and rotated on the way
  attend   every node attends to its request's cached tokens and to its ancestors
  verify   the target's probabilities accept a path of nodes and give the token after it
  compact  the accepted nodes' rows move together in the cache

With `own` false, run() computes them from elementary torch operations; with
`own` true it makes a user's calls of `tl.PagedKVCache` and `tl.tl_verify_tree`.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "fp8": 1}
FP8_MAX = 448.0
EPS = 1e-6
TABLE_ROWS = 131072       # positions that the rotation tables cover


def listed():
    # head layouts: 24 query heads on 4 key-value heads of 256 (the 6-to-1
    # sharing of a 27B model), 40 on 8 of 128 (hidden size 5120)
    big = {"q_heads": 24, "kv_heads": 4, "dim": 256}
    mid = {"q_heads": 40, "kv_heads": 8, "dim": 128}
    return [
        # one person's chat, 8 nodes a step: the latency of one layer counts
        dict(name="attend: one request, 577 tokens", op="attend", batch=1, lo=577, hi=577, few=8, many=8, page=16, type="bf16",
             cache="bf16", window=0, sinks=0, lse=False, padded=0, **big),
        # 24 people at once, each at another point of their conversation, with trees of other sizes, padded to a graph's size
        dict(name="attend: 24 requests, 40 to 9000", op="attend", batch=24, lo=40, hi=9000, few=4, many=26, page=16, type="bf16",
             cache="bf16", window=0, sinks=0, lse=True, padded=24, **big),
        # a loaded server: short drafts over an 8-bit cache, a window and the first tokens
        dict(name="attend: 8-bit, window and sinks", op="attend", batch=160, lo=512, hi=16384, few=1, many=12, page=64, type="f16",
             cache="fp8", window=8192, sinks=4, lse=False, padded=0, **mid),
        # one request with a long document and a broad tree
        dict(name="attend: 80001 tokens, 64 nodes", op="attend", batch=1, lo=80001, hi=80001, few=64, many=64, page=16, type="bf16",
             cache="bf16", window=0, sinks=0, lse=False, padded=0, **big),
        # the trees of one person, and of many people with unlike trees, padded; once a step for all layers
        dict(name="plan: one request, 26 nodes", op="plan", batch=1, lo=700, hi=700, few=26, many=26, page=16, padded=0),
        dict(name="plan: 500 requests", op="plan", batch=500, lo=1, hi=120000, few=1, many=64, page=24, padded=100),
        # one step of 24 people; a quarter of each head is rotated
        dict(name="append: 24 trees of 8", op="append", tokens=192, page=16, type="bf16", cache="bf16", rot=64, interleaved=False,
             norms="qk", padded=0, **big),
        # prompts into an 8-bit cache, neighbours rotated in pairs
        dict(name="append: 16000 prompt tokens", op="append", tokens=16000, page=32, type="f16", cache="fp8", rot=128,
             interleaved=True, norms="qk", padded=37, **mid),
        # one person, a chain of guesses
        dict(name="verify: one chain of 8", op="verify", batch=1, few=8, many=8, vocab=131072, chain=True, drafted=True, near=0.5, padded=0),
        # many people, trees of other sizes, a vocabulary whose rows are not aligned
        dict(name="verify: 64 trees of up to 26", op="verify", batch=64, few=4, many=26, vocab=100001, chain=False, drafted=True,
             near=0.8, padded=9),
        # what verification kept, of one layer: a few rows each, and long chains of a loaded server
        dict(name="compact: 24 requests", op="compact", batch=24, lo=40, hi=2000, kept=4, page=16, cache="bf16", **big),
        dict(name="compact: 160 requests, 8-bit", op="compact", batch=160, lo=100, hi=1000, kept=24, page=64, cache="fp8", **mid),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "plan", "append", "verify", "compact"])
    kind = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = dict(q_heads=kv_heads * rng.choice([1, 2, 4, 5, 6, 7, 8, 12, 16]), kv_heads=kv_heads, dim=dim)
    cache = rng.choice([kind, kind, "fp8"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128, 256])
    many = _log(rng, 1, 64)
    few = _log(rng, 1, many)
    if op == "plan":
        hi = _log(rng, 1, 120000)
        return dict(op=op, batch=_log(rng, 1, 500), lo=_log(rng, 1, hi), hi=hi, few=few, many=many, page=page, padded=rng.randrange(0, 100))
    if op == "append":
        tokens = _log(rng, 1, 16000)
        while tokens * (heads["q_heads"] + 2 * kv_heads) * dim > 16000 * 56 * 128:
            tokens = _log(rng, 1, 16000)
        return dict(op=op, tokens=tokens, page=page, type=kind, cache=cache, rot=rng.choice([0, dim // 4, dim // 2, dim]),
                    interleaved=rng.random() < 0.5, norms=rng.choice(["qk", "qk", "q", "k"]), padded=rng.randrange(0, tokens // 8 + 1), **heads)
    if op == "verify":
        batch, vocab = _log(rng, 1, 64), _log(rng, 1000, 131072)
        while batch * many * vocab > 64 * 26 * 100001:
            batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, few=few, many=many, vocab=vocab, chain=rng.random() < 0.4, drafted=rng.random() < 0.7,
                    near=rng.choice([0.0, 0.5, 0.8, 1.0]), padded=rng.randrange(0, 12))
    if op == "compact":
        hi = _log(rng, 1, 2000)
        batch = _log(rng, 1, 160)
        while batch * (hi + 64) * kv_heads * dim > 160 * 600 * 8 * 128:
            batch = _log(rng, 1, 160)
        return dict(op=op, batch=batch, lo=_log(rng, 1, hi), hi=hi, kept=_log(rng, 1, 32), page=page, cache=cache, **heads)
    batch, hi = _log(rng, 1, 160), _log(rng, 1, 80001)
    while batch * hi * kv_heads * dim > 160 * 4096 * 8 * 128 or batch * hi * many * heads["q_heads"] * dim > 80001 * 64 * 24 * 256:
        batch, hi = _log(rng, 1, 160), _log(rng, 1, 80001)
    window = rng.choice([0, 0, 0, _log(rng, 64, 8192)])
    return dict(op=op, batch=batch, lo=_log(rng, 1, hi), hi=hi, few=few, many=many, page=page, type=kind, cache=cache, window=window,
                sinks=rng.choice([0, 4, 33]) if window else 0, lse=rng.random() < 0.5, padded=rng.randrange(0, 20), **heads)


def _lengths(case):
    """Cached tokens of the batch's requests, spread evenly over their logarithm."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    if b == 1:
        return [hi]
    return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * i / (b - 1)))) for i in range(b)]


def _nodes(case):
    """Nodes of the batch's trees: every size from `few` to `many`, in no order."""
    span = case["many"] - case["few"] + 1
    return [case["few"] + (i * 7919 + span - 1) % span for i in range(case["batch"])]


def _parents(order, nodes, chain):
    """A tree whose parents precede their children; most nodes continue a recent one."""
    return [-1] + [i - 1 if chain else order.randrange(max(0, i - 6), i) for i in range(1, nodes)]


def _masks(parents):
    """Each node's ancestors and itself, as bits of a signed 64-bit number."""
    got = []
    for i, up in enumerate(parents):
        got.append((got[up] if up >= 0 else 0) | 1 << i)
    return [m - (1 << 64) if m >> 63 else m for m in got]


def _ints(values, kind=torch.int32):
    return torch.tensor(values, dtype=kind, device="cuda")


def _forest(s, order, nodes, chain=False):
    """Parents, starts and masks of trees with so many nodes, behind each other."""
    parents = [_parents(order, n, chain) for n in nodes]
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    pad = s["case"].get("padded", 0)
    s["trees"] = parents
    s["total"] = starts[-1] + pad
    s["parents"] = _ints([i for p in parents for i in p] + [-1] * pad)
    s["starts"] = _ints(starts)
    s["masks"] = _ints([m for p in parents for m in _masks(p)] + [0] * pad, torch.int64)


def _normal(gen, shape, kind, outliers=0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if outliers:      # a few channels carry much larger values, as a model's do
        x[..., torch.randperm(shape[-1], generator=gen, device="cuda")[:outliers]] *= 4.0
    return x.to(DTYPES[kind])


def _cache_values(gen, shape, kind, scale):
    """A cache's contents: rotated keys, or values, as stored."""
    out = torch.empty(shape, dtype=DTYPES[kind], device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - i),) + tuple(shape[1:]), generator=gen, device="cuda")
        if kind == "fp8":
            x = (x / scale.view(1, -1, 1, 1)).clamp(-FP8_MAX, FP8_MAX)
        out[i:i + step] = x.to(DTYPES[kind])
    return out


def _table(gen, s, tokens, page):
    """Pages for so many tokens of each request, in random places; returns the number of pages."""
    need = [-(-n // page) for n in tokens]
    pages = sum(need) + 3
    place = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    filled = torch.arange(max(need)).view(1, -1) < torch.tensor(need).view(-1, 1)
    s["pages"] = torch.zeros((len(tokens), max(need)), dtype=torch.int32, device="cuda")
    s["pages"][filled.cuda()] = place[:sum(need)]
    return pages


def _probabilities(gen, rows, vocab, near):
    """Two sets of distributions, the second `near` the first, peaked as a model's are."""
    target, draft = (torch.empty((rows, vocab), device="cuda") for _ in range(2))
    step = max(1, (1 << 27) // vocab)
    for i in range(0, rows, step):
        n = min(step, rows - i)
        x = torch.randn((n, vocab), generator=gen, device="cuda") * 2.5
        y = torch.randn((n, vocab), generator=gen, device="cuda") * 2.5
        target[i:i + n] = torch.softmax(x, 1)
        draft[i:i + n] = torch.softmax(near * x + math.sqrt(1 - near * near) * y, 1)
    return target, draft


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    order = random.Random(seed)
    s = {"case": case}
    op = case["op"]
    if op == "verify":
        _forest(s, order, _nodes(case), case["chain"])
        s["target"], draft = _probabilities(gen, s["total"], case["vocab"], case["near"])
        s["uniform"] = torch.rand((s["total"],), generator=gen, device="cuda")
        # a node's token is drawn from the draft after its parent; without a distribution it is the draft's likeliest
        at = (s["parents"].clamp(min=0) + torch.cat([s["starts"][:-1].repeat_interleave(s["starts"].diff()),
                                                     s["starts"].new_zeros(case["padded"])])).long()
        score = torch.empty((s["total"],), dtype=torch.int64, device="cuda")
        step = max(1, (1 << 27) // case["vocab"])
        for i in range(0, s["total"], step):
            rows = draft[at[i:i + step]]
            e = torch.empty_like(rows).exponential_(generator=gen)
            score[i:i + step] = (rows / e if case["drafted"] else s["target"][at[i:i + step]] / e.clamp(min=0.3)).argmax(1)
        s["tokens"] = score.int()
        s["draft"] = draft if case["drafted"] else None
        s["path"], s["counts"], s["next"] = (torch.empty((n,), dtype=torch.int32, device="cuda") for n in (s["total"], case["batch"], case["batch"]))
        return s

    page = case["page"]
    if op == "plan":
        pairs = list(zip(_lengths(case), _nodes(case)))
        order.shuffle(pairs)
        s["lens"] = _ints([n for n, _ in pairs])
        _forest(s, order, [n for _, n in pairs])
        pages = _table(gen, s, [a + b for a, b in pairs], page)
        s["k"] = s["v"] = torch.zeros((pages, 1, page, 16), dtype=torch.bfloat16, device="cuda")
        s["got"] = [torch.empty((s["total"],), dtype=k, device="cuda") for k in (torch.int64, torch.int32, torch.int64)]
        if own:
            from quantized_linear_layers_block_gb300 import tl
            s["kv"] = tl.PagedKVCache(pages, page, 1, 16, k=s["k"], v=s["v"])
        return s

    kv_heads, dim = case["kv_heads"], case["dim"]
    scales = [0.02 + 0.01 * torch.rand((kv_heads,), generator=gen, device="cuda") for _ in range(2)] if case["cache"] == "fp8" else [None, None]
    if op == "attend":
        pairs = list(zip(_lengths(case), _nodes(case)))
        order.shuffle(pairs)
        s["lens"] = _ints([n for n, _ in pairs])
        _forest(s, order, [n for _, n in pairs])
        pages = _table(gen, s, [a + b for a, b in pairs], page)
        s["q"] = _normal(gen, (s["total"], case["q_heads"], dim), case["type"])
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((s["total"], case["q_heads"]), device="cuda") if case["lse"] else None
    elif op == "compact":
        lens = _lengths(case)
        order.shuffle(lens)
        # request i keeps 1 to `kept` nodes; its tree has them behind the places that they move to
        kept = [1 + i % case["kept"] for i in range(case["batch"])]
        paths = [[0] + sorted(order.sample(range(n, 64), n - 1)) for n in kept]
        s["lens"], s["counts"] = _ints(lens), _ints(kept)
        s["starts"] = _ints([64 * i for i in range(case["batch"] + 1)])
        s["path"] = _ints([j for p in paths for j in p + [-1] * (64 - len(p))])
        pages = _table(gen, s, [n + 64 for n in lens], page)
    else:
        t, heads = case["tokens"], case["q_heads"]
        pages = -(-(t + 40) // page) + 2
        # queries, keys and values lie side by side, as a fused projection writes them
        qkv = _normal(gen, (t, (heads + 2 * kv_heads) * dim), case["type"], outliers=4)
        s["q"] = qkv[:, :heads * dim].view(t, heads, dim)
        s["k_new"] = qkv[:, heads * dim:(heads + kv_heads) * dim].view(t, kv_heads, dim)
        s["v_new"] = qkv[:, (heads + kv_heads) * dim:].view(t, kv_heads, dim)
        s["q_out"] = torch.empty((t, heads, dim), dtype=qkv.dtype, device="cuda")
        for n in "qk":
            s[n + "_norm"] = 1.0 + 0.2 * torch.randn((dim,), generator=gen, device="cuda") if n in case["norms"] else None
        start = order.randrange(0, TABLE_ROWS - t)
        s["positions"] = torch.arange(start, start + t, dtype=torch.int32, device="cuda")
        slots = torch.randperm(pages, generator=gen, device="cuda").repeat_interleave(page) * page
        slots = (slots + torch.arange(page, device="cuda").repeat(pages))[:t].clone()
        if case["padded"]:
            slots[t - case["padded"]:] = -1
        s["slots"] = slots.to(torch.int64)
        s["cos_sin"] = None
        if case["rot"]:
            half = case["rot"] // 2
            rate = torch.pow(10000.0, -torch.arange(half, dtype=torch.float64, device="cuda") / half)
            angle = torch.arange(TABLE_ROWS, dtype=torch.float64, device="cuda").view(-1, 1) * rate
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    s["k"] = _cache_values(gen, (pages, kv_heads, page, dim), case["cache"], scales[0])
    s["v"] = _cache_values(gen, (pages, kv_heads, page, dim), case["cache"], scales[1])
    s["k_scale"], s["v_scale"] = scales
    if own:
        from quantized_linear_layers_block_gb300 import tl
        s["kv"] = tl.PagedKVCache(pages, page, kv_heads, dim, dtype=DTYPES[case["cache"]], k_scale=scales[0], v_scale=scales[1], k=s["k"], v=s["v"])
    return s


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"plan": _plan, "append": _append, "attend": _attend, "verify": _verify, "compact": _compact}[op](s)
    if op == "plan":
        masks, positions, slots = s["kv"].plan_tree(s["parents"], s["starts"], s["lens"], s["pages"], masks=s["got"][0], positions=s["got"][1],
                                                    slots=s["got"][2])
        return {"masks": masks, "positions": positions, "slots": slots}
    if op == "append":
        q = s["kv"].append(s["k_new"], s["v_new"], s["positions"], s["slots"], cos_sin=s["cos_sin"], interleaved=c["interleaved"],
                           q=s["q"], q_out=s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return {"q": q, "k": s["k"], "v": s["v"]}
    if op == "attend":
        out = s["kv"].attend_tree(s["q"], s["masks"], s["starts"], s["pages"], s["lens"], window=c["window"], sinks=c["sinks"],
                                  out=s["out"], lse=s["lse"])
        return {"out": out} if s["lse"] is None else {"out": out, "lse": s["lse"]}
    if op == "verify":
        from quantized_linear_layers_block_gb300 import tl
        path, counts, after = tl.tl_verify_tree(s["target"], s["draft"], s["tokens"], s["parents"], s["starts"], s["uniform"],
                                                path=s["path"], counts=s["counts"], next=s["next"])
        return {"path": path, "counts": counts, "next": after}
    s["kv"].compact(s["path"], s["counts"], s["starts"], s["pages"], s["lens"])
    return {"k": s["k"], "v": s["v"]}


def _boxed(s):
    """For each request and each of 64 places: is there a node, and which row has it."""
    begin, n = s["starts"][:-1].long().view(-1, 1), s["starts"].diff().long().view(-1, 1)
    at = torch.arange(64, device="cuda").view(1, -1)
    return at < n, torch.where(at < n, begin + at, 0)


def _plan(s):
    there, rows = _boxed(s)
    up = torch.where(there, s["parents"][rows].long(), -1)
    at = torch.arange(64, device="cuda")
    # who is reached in one step or none, then in up to 2, 4, ... 64
    reach = ((up.unsqueeze(2) == at) | torch.eye(64, dtype=torch.bool, device="cuda")).float()
    for _ in range(6):
        reach = (torch.matmul(reach, reach) > 0).float()
    bits = (reach > 0) & there.unsqueeze(2)
    word = torch.ones((), dtype=torch.int64, device="cuda") << at
    masks = torch.zeros((s["total"],), dtype=torch.int64, device="cuda")
    positions = torch.zeros((s["total"],), dtype=torch.int32, device="cuda")
    slots = torch.full((s["total"],), -1, dtype=torch.int64, device="cuda")
    masks[rows[there]] = (bits * word).sum(2)[there]
    positions[rows[there]] = (s["lens"].view(-1, 1) + bits.sum(2) - 1).int()[there]
    page = s["case"]["page"]
    key = s["lens"].view(-1, 1).long() + at
    pages = torch.gather(s["pages"].long(), 1, (key // page).clamp(max=s["pages"].shape[1] - 1))
    slots[rows[there]] = (pages * page + key % page)[there]
    return {"masks": masks, "positions": positions, "slots": slots}


def _turned(x, cos, sin, rot, interleaved):
    """x [tokens, heads, dim] with its first `rot` channels rotated by the angles of cos and sin [tokens, rot / 2]."""
    if not rot:
        return x
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    r = x[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _normed(x, weight):
    return x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _angles(s, wide=False):
    rot = s["case"]["rot"]
    if not rot:
        return None, None
    rows = s["cos_sin"][s["positions"].long()]
    rows = rows.double() if wide else rows
    return rows[:, :rot // 2], rows[:, rot // 2:]


def _stored(cache, rows, slots, page, scale):
    """Writes rows [tokens, heads, dim] to their slots of the cache."""
    if scale is not None:
        rows = (rows * (1.0 / scale).view(1, -1, 1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache = cache.view(torch.uint8)
    else:
        rows = rows.to(cache.dtype)
    kept = slots >= 0
    at = slots[kept]
    cache[at // page, :, at % page] = rows[kept]


def _append(s):
    c = s["case"]
    cos, sin = _angles(s)
    q = _turned(_normed(s["q"].float(), s["q_norm"]), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    k = _turned(_normed(s["k_new"].float(), s["k_norm"]), cos, sin, c["rot"], c["interleaved"])
    _stored(s["k"], k, s["slots"], c["page"], s["k_scale"])
    _stored(s["v"], s["v_new"].float(), s["slots"], c["page"], s["v_scale"])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _gathered(cache, table, kind):
    """[pages, heads, page, dim] by a table [batch, pages] -> [batch, heads, pages * page, dim] in 32 bits."""
    bits = cache.view(torch.uint8) if kind == "fp8" else cache
    rows = bits[table.long()]
    rows = (rows.view(torch.float8_e4m3fn) if kind == "fp8" else rows).float()
    b, n, h, p, d = rows.shape
    return rows.permute(0, 2, 1, 3, 4).reshape(b, h, n * p, d)


def _seen(s, most, keys):
    """[batch, most, keys]: which keys each node sees."""
    c = s["case"]
    there, rows = _boxed(s)
    masks = torch.where(there, s["masks"][rows], 0)[:, :most].unsqueeze(2)
    bits = (masks >> torch.arange(64, device="cuda")) & 1
    at = torch.arange(keys, device="cuda").view(1, 1, -1)
    n = s["lens"].long().view(-1, 1, 1)
    seen = at < n
    if c["window"]:
        seen = seen & ((at >= n - (c["window"] - bits.sum(2, keepdim=True)).clamp(min=0)) | (at < c["sinks"]))
    node = (at - n).expand(-1, most, -1)
    drafted = torch.gather(bits, 2, node.clamp(0, 63)) > 0
    return torch.where(node < 0, seen, drafted & (node < 64))


def _attend(s):
    c = s["case"]
    b, hq, hkv, d, most = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["many"]
    there, rows = _boxed(s)
    there, rows = there[:, :most], rows[:, :most]
    q = s["q"].float()[rows].view(b, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    k = _gathered(s["k"], s["pages"], c["cache"])
    if s["k_scale"] is not None:
        k *= s["k_scale"].view(1, -1, 1, 1)
    x = (torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))).view(b, hkv, hq // hkv, most, -1)
    del k
    seen = _seen(s, most, x.shape[4])
    x = torch.where(seen.view(b, 1, 1, most, -1), x, -math.inf)
    top = x.amax(4, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(x - top)
    del x
    total = p.sum(4, keepdim=True)
    v = _gathered(s["v"], s["pages"], c["cache"])
    if s["v_scale"] is not None:
        v *= s["v_scale"].view(1, -1, 1, 1)
    y = torch.matmul(p.view(b, hkv, -1, p.shape[4]), v).view(b, hkv, hq // hkv, most, d) / torch.where(total > 0, total, 1.0)
    out = torch.zeros_like(s["q"])
    out[rows[there]] = y.permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)[there].to(out.dtype)
    if s["lse"] is None:
        return {"out": out}
    lse = torch.zeros_like(s["lse"])
    lse[rows[there]] = (top + torch.log(total)).permute(0, 3, 1, 2, 4).reshape(b, most, hq)[there]
    return {"out": out, "lse": lse}


def _verify(s):
    """All requests at once, in 64 bits, node after node: a node whose parent is where its request stands is tried."""
    c = s["case"]
    b = c["batch"]
    there, rows = _boxed(s)
    at = torch.zeros((b,), dtype=torch.int64, device="cuda")           # where each request stands
    left = s["target"][rows[:, 0]].double()                            # what is left of the distribution there
    total = torch.ones((b,), dtype=torch.float64, device="cuda")
    count = torch.ones_like(at)
    path = torch.full((s["total"],), -1, dtype=torch.int32, device="cuda")
    path[rows[:, 0]] = 0
    for i in range(1, c["many"]):
        row = rows[:, i]
        here = there[:, i] & (s["parents"][row] == at)
        token = s["tokens"][row].long().view(-1, 1)
        where = torch.gather(rows, 1, at.view(-1, 1)).view(-1)
        if s["draft"] is None:
            q = torch.zeros_like(left).scatter_(1, token, 1.0)
        else:
            q = s["draft"][where].double()
        p = torch.gather(left, 1, token).view(-1)
        taken = here & (s["uniform"][row].double() * torch.gather(q, 1, token).view(-1) * total < p)
        missed = here & ~taken
        rest = (left - total.view(-1, 1) * q).clamp(min=0)
        left = torch.where(missed.view(-1, 1), rest, torch.where(taken.view(-1, 1), s["target"][row].double(), left))
        total = torch.where(missed, rest.sum(1), torch.where(taken, 1.0, total))
        place = torch.gather(rows, 1, count.view(-1, 1)).view(-1)
        path[torch.where(taken, place, rows[:, 0])] = torch.where(taken, i, 0).int()
        count += taken
        at = torch.where(taken, i, at)
    sums = left.cumsum(1)
    none = sums[:, -1:] <= 0          # nothing is left: the target's own
    sums = torch.where(none, s["target"][torch.gather(rows, 1, at.view(-1, 1)).view(-1)].double().cumsum(1), sums)
    after = (sums <= s["uniform"][rows[:, 0]].double().view(-1, 1) * sums[:, -1:]).sum(1).clamp(max=c["vocab"] - 1)
    return {"path": path, "counts": count.int(), "next": after.int()}


def _compact(s):
    c = s["case"]
    path = s["path"].view(-1, 64).long()
    to = torch.arange(64, device="cuda").view(1, -1)
    moved = (to < s["counts"].view(-1, 1)) & (path != to)
    page, n = c["page"], s["lens"].long().view(-1, 1)
    for name in ("k", "v"):
        cache = s[name].view(torch.uint8) if c["cache"] == "fp8" else s[name]
        source, place = (torch.gather(s["pages"].long(), 1, key // page)[moved] for key in (n + path.clamp(min=0), n + to))
        cache[place, :, ((n + to) % page)[moved]] = cache[source, :, ((n + path.clamp(min=0)) % page)[moved]]
    return {"k": s["k"], "v": s["v"]}


def work(case):
    op = case["op"]
    if op == "verify":
        # a request's last distribution is read whole, with the draft's where one of its guesses was refused
        v = case["batch"] * case["vocab"]
        return {"bytes": v * (8 if case["drafted"] else 4) + 16 * sum(_nodes(case)), "flops": 3 * v}
    if op == "plan":
        t = sum(_nodes(case)) + case["padded"]
        return {"bytes": t * (4 + 8 + 4 + 8) + case["batch"] * 16, "flops": 64 * t}
    hkv, d = case["kv_heads"], case["dim"]
    ec = BYTES[case["cache"]]
    if op == "compact":
        moved = sum(i % case["kept"] for i in range(case["batch"]))
        return {"bytes": max(1, 4 * moved * hkv * d * ec), "flops": 0}
    hq, e = case["q_heads"], BYTES[case["type"]]
    if op == "append":
        t, kept = case["tokens"], case["tokens"] - case["padded"]
        return {"bytes": 2 * t * hq * d * e + 2 * kept * hkv * d * (e + ec) + t * (4 * case["rot"] + 12) + 8 * d,
                "flops": (3 * case["rot"] + 4 * d) * (t * hq + kept * hkv)}
    keys, pairs = 0, 0
    for n, m in zip(_lengths(case), _nodes(case)):
        cached = min(n, case["window"] + case["sinks"]) if case["window"] else n
        keys += cached + m
        pairs += cached * m + m * (m + 1) // 4
    t = sum(_nodes(case))
    return {"bytes": 2 * keys * hkv * d * ec + 2 * t * hq * d * e + 4 * (keys // case["page"] + case["batch"]) + 8 * t, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    """The operators in 64 bits, request by request."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"plan": _exact_plan, "append": _exact_append, "attend": _exact_attend, "verify": _exact_verify, "compact": _exact_compact}[case["op"]](s)


def _exact_plan(s):
    page, table, lens = s["case"]["page"], s["pages"].tolist(), s["lens"].tolist()
    masks, positions, slots = [], [], []
    for b, tree in enumerate(s["trees"]):
        depth = []
        for i, up in enumerate(tree):
            depth.append(0 if up < 0 else depth[up] + 1)
            positions.append(lens[b] + depth[i])
            slots.append(table[b][(lens[b] + i) // page] * page + (lens[b] + i) % page)
        masks += _masks(tree)
    pad = s["total"] - len(masks)
    return {"masks": _ints(masks + [0] * pad, torch.int64), "positions": _ints(positions + [0] * pad), "slots": _ints(slots + [-1] * pad, torch.int64)}


def _exact_append(s):
    case = s["case"]
    at, t, page = s["slots"].tolist(), case["tokens"], case["page"]
    cos, sin = _angles(s, wide=True)
    res, rot, half = {}, case["rot"], case["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    kept = torch.tensor([i for i in range(t) if at[i] >= 0], dtype=torch.int64, device="cuda")
    for name, new, scale in (("q", "q", None), ("k", "k_new", "k_scale"), ("v", "v_new", "v_scale")):
        x = s[new].double()
        if name != "v" and s[name + "_norm"] is not None:
            x = x * torch.rsqrt(x.pow(2).sum(2, keepdim=True) / case["dim"] + EPS) * s[name + "_norm"].double()
        if rot and name != "v":
            z = torch.complex(x[..., first], x[..., second]) * torch.complex(cos, sin).unsqueeze(1)
            x[..., first], x[..., second] = z.real, z.imag
        if name == "q":
            res["q"] = x
            continue
        full = s[name].double()
        rows = x[kept]
        if s[scale] is not None:
            rows = (rows / s[scale].double().view(1, -1, 1)).clamp(-FP8_MAX, FP8_MAX)
        where = s["slots"][kept]
        full[where // page, :, where % page] = rows
        res[name] = full
    return res


def _exact_attend(s):
    case = s["case"]
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.zeros((s["total"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], hq), dtype=torch.float64, device="cuda")
    row = 0
    for b, n in enumerate(s["lens"].tolist()):
        tree = _masks(s["trees"][b])
        m = len(tree)
        keys = range(max(0, n - case["window"]), n + m) if case["window"] else range(n + m)
        at = torch.tensor(sorted(set(range(min(n, case["sinks"]))) | set(keys)), device="cuda")
        where = s["pages"][b].long()[at // page]
        rows = []
        for name, scale in (("k", "k_scale"), ("v", "v_scale")):
            x = s[name].view(torch.uint8)[where, :, at % page].view(torch.float8_e4m3fn) if case["cache"] == "fp8" else s[name][where, :, at % page]
            x = x.double().transpose(0, 1)
            rows.append(x if s[scale] is None else x * s[scale].double().view(-1, 1, 1))
        sees = torch.zeros((m, len(at)), dtype=torch.bool, device="cuda")
        for i, word in enumerate(tree):
            nodes = [j for j in range(m) if word >> j & 1]
            back = max(0, case["window"] - len(nodes)) if case["window"] else n
            sees[i] = (at < n) & ((at >= n - back) | (at < case["sinks"]))
            sees[i] |= torch.isin(at, _ints([n + j for j in nodes], torch.int64))
        q = s["q"][row:row + m].double().view(m, hkv, hq // hkv, d)
        z = torch.einsum("mhgd,hnd->hgmn", q, rows[0]) / math.sqrt(d)
        z = z.masked_fill(~sees, -math.inf)
        lse[row:row + m] = torch.logsumexp(z, 3).permute(2, 0, 1).reshape(m, hq)
        out[row:row + m] = torch.einsum("hgmn,hnd->mhgd", torch.softmax(z, 3), rows[1]).reshape(m, hq, d)
        row += m
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_verify(s):
    parents, tokens, uniform = s["trees"], s["tokens"].tolist(), s["uniform"].double().tolist()
    path, counts, after = [-1] * s["total"], [], []
    row = 0
    for tree in parents:
        node, way = 0, [0]
        while True:
            p = s["target"][row + node].double()
            found = None
            for child in [i for i, up in enumerate(tree) if up == node]:
                x = tokens[row + child]
                q = torch.zeros_like(p) if s["draft"] is None else s["draft"][row + node].double()
                if s["draft"] is None:
                    q[x] = 1.0
                if uniform[row + child] * float(q[x]) < float(p[x]):
                    found = child
                    break
                p = torch.clamp(p - q, min=0)
                p = p / p.sum() if float(p.sum()) > 0 else p
            if found is None:
                break
            node = found
            way.append(node)
        p = p if float(p.sum()) > 0 else s["target"][row + node].double()
        sums = torch.cumsum(p, 0)
        after.append(min(int(torch.searchsorted(sums, uniform[row] * sums[-1], right=True)), p.numel() - 1))
        counts.append(len(way))
        path[row:row + len(way)] = way
        row += len(tree)
    return {"path": _ints(path), "counts": _ints(counts), "next": _ints(after)}


def _exact_compact(s):
    page, lens, counts = s["case"]["page"], s["lens"].tolist(), s["counts"].tolist()
    path, table = s["path"].tolist(), s["pages"].tolist()
    res = {}
    for name in ("k", "v"):
        full = s[name].double()
        moves = [(b, n + path[64 * b + j], n + j) for b, n in enumerate(lens) for j in range(counts[b])]
        source = _ints([table[b][x // page] * page + x % page for b, x, _ in moves], torch.int64)
        place = _ints([table[b][y // page] * page + y % page for b, _, y in moves], torch.int64)
        full[place // page, :, place % page] = full[source // page, :, source % page].clone()
        res[name] = full
    return res
