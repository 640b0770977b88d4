"""What is measured of the operators that serve the attention half of a decoder layer for many requests.

Three operators stand between and beside the ternary projections of such a layer:

  append   new tokens' keys and values go into a paged cache, rotated by their
           positions on the way; the queries are rotated by the same call
  attend   one new token of each request attends to its cached keys and values
  adapt    every token's low-rank adapter is added to a projection's output

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true it makes a user's calls of `tl.PagedKVCache` and
`tl.LoraBank`.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
FP8_MAX = 448.0
TABLE_ROWS = 32768        # positions that the rotation tables cover


def listed():
    # head layouts: 24 query heads on 4 key-value heads of 256 (the 6-to-1
    # sharing of a 27B model), 40 on 8 of 128 (hidden size 5120), 16 on 16 of 64
    big = {"q_heads": 24, "kv_heads": 4, "dim": 256}
    mid = {"q_heads": 40, "kv_heads": 8, "dim": 128}
    small = {"q_heads": 16, "kv_heads": 16, "dim": 64}
    return [
        # a single chat turn early in its life: the latency of one layer counts
        dict(name="attend: one request, 577 tokens", op="attend", batch=1, lo=577, hi=577, page=16, type="bf16", cache="bf16",
             window=0, lse=False, **big),
        # 24 people at once, each at another point of their conversation
        dict(name="attend: 24 requests, 40 to 9000", op="attend", batch=24, lo=40, hi=9000, page=16, type="bf16", cache="bf16",
             window=0, lse=True, **big),
        # one request with a long document in its context
        dict(name="attend: one request, 80001 tokens", op="attend", batch=1, lo=80001, hi=80001, page=16, type="bf16", cache="bf16",
             window=0, lse=False, **big),
        # a sliding-window layer without head sharing, with pages that are no power of two, and very short requests
        dict(name="attend: window 1024, 96 requests", op="attend", batch=96, lo=1, hi=6000, page=24, type="f16", cache="f16",
             window=1024, lse=False, **small),
        # a loaded server with an 8-bit cache
        dict(name="attend: 8-bit cache, 160 requests", op="attend", batch=160, lo=512, hi=16384, page=64, type="bf16", cache="fp8",
             window=0, lse=False, **mid),
        # one decode step of 24 people; a quarter of each head is rotated
        dict(name="append: 24 new tokens", op="append", tokens=24, page=16, type="bf16", cache="bf16", rot=64, interleaved=False,
             padded=0, **big),
        # one chunk of a prompt into an 8-bit cache, neighbours rotated in pairs, padded to the chunk size
        dict(name="append: 512-token chunk, 8-bit", op="append", tokens=512, page=64, type="bf16", cache="fp8", rot=128,
             interleaved=True, padded=37, **mid),
        # many prompts at once
        dict(name="append: 16000 prompt tokens", op="append", tokens=16000, page=32, type="f16", cache="f16", rot=128,
             interleaved=False, padded=0, **mid),
        # one token of one request beside the gate projection
        dict(name="adapt: 1 token, rank 16", op="adapt", tokens=1, inner=5120, outer=17408, rank=16, adapters=8, bare=0, type="bf16",
             out="bf16"),
        # a decode batch in which nearly everybody has an adapter of their own
        dict(name="adapt: 48 tokens, 32 adapters", op="adapt", tokens=48, inner=5120, outer=5120, rank=32, adapters=32, bare=5,
             type="bf16", out="bf16"),
        # a prompt chunk of several requests beside the down projection, in 32-bit outputs
        dict(name="adapt: 515 tokens, rank 64", op="adapt", tokens=515, inner=17408, outer=5120, rank=64, adapters=5, bare=3,
             type="f16", out="f32"),
        # long prompts beside the fused gate and up projection
        dict(name="adapt: 4096 prompt tokens", op="adapt", tokens=4096, inner=5120, outer=34816, rank=16, adapters=3, bare=0,
             type="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "adapt"])
    kind = rng.choice(["bf16", "f16"])
    if op == "adapt":
        tokens = _log(rng, 1, 4096)
        inner = 8 * _log(rng, 64, 2176)
        outer = 8 * _log(rng, 64, 4352)
        while tokens * outer > 4096 * 34816:
            outer = 8 * _log(rng, 64, 4352)
        return dict(op=op, tokens=tokens, inner=inner, outer=outer, rank=rng.choice([8, 16, 32, 64, 128]),
                    adapters=_log(rng, 1, 48), bare=rng.randrange(0, tokens // 8 + 1), type=kind,
                    out=rng.choice([kind, kind, "f32"]))
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = dict(q_heads=kv_heads * rng.choice([1, 2, 4, 5, 6, 7, 8, 12, 16]), kv_heads=kv_heads, dim=dim)
    cache = rng.choice([kind, kind, "fp8"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 128, 256])
    if op == "append":
        tokens = _log(rng, 1, 16000)
        while tokens * (heads["q_heads"] + 2 * kv_heads) * dim > 16000 * 56 * 128:
            tokens = _log(rng, 1, 16000)
        return dict(op=op, tokens=tokens, page=page, type=kind, cache=cache, rot=rng.choice([0, dim // 4, dim // 2, dim]),
                    interleaved=rng.random() < 0.5, padded=rng.randrange(0, tokens // 8 + 1), **heads)
    batch = _log(rng, 1, 160)
    hi = _log(rng, 1, 80001)
    while batch * hi * kv_heads * dim > 160 * 4096 * 8 * 128:
        batch, hi = _log(rng, 1, 160), _log(rng, 1, 80001)
    return dict(op=op, batch=batch, lo=_log(rng, 1, hi), hi=hi, page=page, type=kind, cache=cache,
                window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), lse=rng.random() < 0.5, **heads)


def _lengths(case):
    """Lengths of the batch's requests, spread evenly over their logarithm."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    if b == 1:
        return [hi]
    return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * i / (b - 1)))) for i in range(b)]


def _seen(case):
    """Cached tokens that each request's new token attends to."""
    return [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]


def _normal(gen, shape, kind, outliers=0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if outliers:      # a few channels carry much larger values, as a model's do
        at = torch.randperm(shape[-1], generator=gen, device="cuda")[:outliers]
        x[..., at] *= 4.0
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    order = random.Random(seed)
    s = {"case": case}
    if case["op"] == "adapt":
        m, k, n, r, na = (case[i] for i in ("tokens", "inner", "outer", "rank", "adapters"))
        s["x"] = _normal(gen, (m, k), case["type"], outliers=4)
        s["base"] = _normal(gen, (m, n), case["out"])
        s["A"] = (torch.randn((na, r, k), generator=gen, device="cuda") / math.sqrt(k)).to(DTYPES[case["type"]])
        s["B"] = (torch.randn((na, n, r), generator=gen, device="cuda") / math.sqrt(r)).to(DTYPES[case["type"]])
        s["scale"] = 0.5 + torch.rand((na,), generator=gen, device="cuda")
        # requests come in runs of tokens, each with one adapter, at most two runs of the same; -1: none
        cuts = sorted(order.sample(range(1, m), min(m, 2 * na) - 1))
        turns = order.sample(range(na), na) + order.sample(range(na), na)
        ids = [a for a, begin, end in zip(turns, [0] + cuts, cuts + [m]) for _ in range(end - begin)]
        for i in order.sample(range(m), case["bare"]):
            ids[i] = -1
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty_like(s["base"])
        if own:
            from quantized_linear_layers_block_gb300 import tl
            s["bank"] = tl.LoraBank(s["A"], s["B"], s["scale"])
            s["plan"] = s["bank"].plan(s["ids"])
        return s

    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    scales = [0.02 + 0.01 * torch.rand((hkv,), generator=gen, device="cuda") for _ in range(2)] if case["cache"] == "fp8" else [None, None]
    if case["op"] == "attend":
        lens = _lengths(case)
        order.shuffle(lens)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        place = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
        table = torch.zeros((case["batch"], max(need)), dtype=torch.int32)
        filled = torch.arange(max(need)).view(1, -1) < torch.tensor(need).view(-1, 1)
        table = table.cuda()
        table[filled.cuda()] = place[:sum(need)]
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _normal(gen, (case["batch"], hq, d), case["type"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["batch"], hq), device="cuda") if case["lse"] else None
    else:
        t = case["tokens"]
        pages = -(-(t + 40) // page) + 2
        # queries, keys and values lie side by side, as a fused projection writes them
        qkv = _normal(gen, (t, (hq + 2 * hkv) * d), case["type"])
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k_new"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v_new"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        s["q_out"] = torch.empty((t, hq, d), dtype=qkv.dtype, device="cuda")
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
    s["k"] = _cache_values(gen, (pages, hkv, page, d), case["cache"], scales[0])
    s["v"] = _cache_values(gen, (pages, hkv, page, d), case["cache"], scales[1])
    s["k_scale"], s["v_scale"] = scales
    if own:
        from quantized_linear_layers_block_gb300 import tl
        s["kv"] = tl.PagedKVCache(pages, page, hkv, d, dtype=DTYPES[case["cache"]], k_scale=scales[0], v_scale=scales[1], k=s["k"], v=s["v"])
    return s


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attend": _attend, "append": _append, "adapt": _adapt}[op](s)
    if op == "attend":
        out = s["kv"].attend(s["q"], s["table"], s["lens"], window=s["case"]["window"], out=s["out"], lse=s["lse"])
        return {"out": out} if s["lse"] is None else {"out": out, "lse": s["lse"]}
    if op == "append":
        q = s["kv"].append(s["k_new"], s["v_new"], s["positions"], s["slots"], cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"],
                           q=s["q"], q_out=s["q_out"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    return {"y": s["bank"].apply(s["x"], s["base"], s["plan"], out=s["out"])}


def _gathered(cache, table, kind):
    """[pages, heads, page, dim] by a table [batch, pages] -> [batch, heads, pages * page, dim] in 32 bits."""
    bits = cache.view(torch.uint8) if kind == "fp8" else cache
    rows = bits[table.long()]
    rows = (rows.view(torch.float8_e4m3fn) if kind == "fp8" else rows).float()
    b, n, h, p, d = rows.shape
    return rows.permute(0, 2, 1, 3, 4).reshape(b, h, n * p, d)


def _attend(s):
    c = s["case"]
    b, hq, hkv, d = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    k = _gathered(s["k"], s["table"], c["cache"])
    if s["k_scale"] is not None:
        k *= s["k_scale"].view(1, -1, 1, 1)
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    at = torch.arange(x.shape[3], device=x.device).view(1, 1, 1, -1)
    n = s["lens"].view(-1, 1, 1, 1)
    seen = at < n
    if c["window"]:
        seen = seen & (at >= n - c["window"])
    x = torch.where(seen, x, -math.inf)
    top = x.amax(3, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(x - top)
    total = p.sum(3, keepdim=True)
    v = _gathered(s["v"], s["table"], c["cache"])
    if s["v_scale"] is not None:
        v *= s["v_scale"].view(1, -1, 1, 1)
    y = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    out = {"out": y.reshape(b, hq, d).to(s["q"].dtype)}
    if c["lse"]:
        out["lse"] = (top + torch.log(total)).reshape(b, hq)
    return out


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
    q = _turned(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    k = _turned(s["k_new"].float(), cos, sin, c["rot"], c["interleaved"])
    _stored(s["k"], k, s["slots"], c["page"], s["k_scale"])
    _stored(s["v"], s["v_new"].float(), s["slots"], c["page"], s["v_scale"])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _adapt(s):
    c = s["case"]
    na, r = c["adapters"], c["rank"]
    mine = s["ids"].view(-1, 1) == torch.arange(na, device="cuda", dtype=torch.int32).view(1, -1)
    h = torch.matmul(s["x"].float(), s["A"].float().view(na * r, -1).t()).view(-1, na, r)
    h = h * (mine.float() * s["scale"]).unsqueeze(2)
    d = torch.matmul(h.view(-1, na * r), s["B"].float().transpose(1, 2).reshape(na * r, -1))
    return {"y": (s["base"].float() + d).to(s["base"].dtype)}


def work(case):
    if case["op"] == "adapt":
        m, k, n, r = case["tokens"], case["inner"], case["outer"], case["rank"]
        live = m - case["bare"]
        used = min(case["adapters"], live)
        e = BYTES[case["type"]]
        return {"bytes": live * k * e + used * r * (k + n) * e + 2 * m * n * BYTES[case["out"]], "flops": 2 * live * r * (k + n)}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    e, ec = BYTES[case["type"]], BYTES[case["cache"]]
    if case["op"] == "append":
        t, kept = case["tokens"], case["tokens"] - case["padded"]
        return {"bytes": 2 * t * hq * d * e + 2 * kept * hkv * d * (e + ec) + t * (4 * case["rot"] + 12),
                "flops": 3 * case["rot"] * (t * hq + kept * hkv)}
    seen = sum(_seen(case))
    return {"bytes": 2 * seen * hkv * d * ec + 2 * case["batch"] * hq * d * e + 4 * (seen // case["page"] + case["batch"]),
            "flops": 4 * seen * hq * d}


def exact(case, seed):
    """The operators in 64 bits, request by request and adapter by adapter."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "adapt":
        y = s["base"].double()
        ids = s["ids"].tolist()
        for a in sorted(set(ids) - {-1}):
            rows = torch.tensor([i for i, b in enumerate(ids) if b == a], device="cuda")
            h = s["x"][rows].double() @ s["A"][a].double().t()
            y[rows] += s["scale"][a].double() * (h @ s["B"][a].double().t())
        return {"y": y}
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        at, t = s["slots"].tolist(), case["tokens"]
        cos, sin = _angles(s, wide=True)
        res, rot, half = {}, case["rot"], case["rot"] // 2
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        kept = torch.tensor([i for i in range(t) if at[i] >= 0], dtype=torch.int64, device="cuda")
        for name, new, scale in (("q", "q", None), ("k", "k_new", "k_scale"), ("v", "v_new", "v_scale")):
            x = s[new].double()
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
    out = torch.empty((case["batch"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((case["batch"], hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        begin = max(0, n - case["window"]) if case["window"] else 0
        ids = s["table"][b, begin // page:-(-n // page)].long()
        lo = begin - begin // page * page
        rows = []
        for name, scale in (("k", "k_scale"), ("v", "v_scale")):
            x = s[name]
            x = x.view(torch.uint8)[ids].view(torch.float8_e4m3fn) if case["cache"] == "fp8" else x[ids]
            x = x.transpose(0, 1).reshape(hkv, -1, d)[:, lo:lo + n - begin].double()
            rows.append(x if s[scale] is None else x * s[scale].double().view(-1, 1, 1))
        z = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(hkv, hq // hkv, d), rows[0]) / math.sqrt(d)
        lse[b] = torch.logsumexp(z, 2).reshape(-1)
        out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(z, 2), rows[1]).reshape(hq, d)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
