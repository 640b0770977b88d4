"""GPU parity of tl_kv_append: bit for bit the fp32 formula of the oracle
(oracle/serving.py), each product and sum rounded on its own, rounded once to the
stored type; and within that type's half unit in the last place of the 64-bit formula."""

import numpy as np
import pytest
import torch

from oracle import serving as O
from quantized_linear_layers_block_gb300 import tl

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}


def angles(max_pos, rot):
    half = rot // 2
    a = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(half) / max(half, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def case(T, hq, hkv, d, page, dtype="bf16", cache=None, rot=None, interleaved=False, layout="heads", padded=(), seed=0, fused=True,
         in_place=False, spread=1.0):
    rng = np.random.default_rng(seed)
    cache = cache or dtype
    rot = d if rot is None else rot
    dt, ct = TYPES[dtype], TYPES[cache]
    pages = -(-T // page) + 3
    width = (hq + 2 * hkv) * d
    qkv = (torch.tensor(rng.standard_normal((T, width + (64 if fused else 0))).astype(np.float32)) * spread).to(dt)
    q, k, v = (qkv[:, a * d:b * d].reshape(T, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    dev = qkv.cuda()
    qd, kd, vd = (dev[:, a * d:b * d].unflatten(1, (b - a, d)) if b > a else dev[:, :0].reshape(T, 0, d)
                  for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    cs = angles(500, rot)
    pos = rng.integers(0, 500, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[list(padded)] = -1
    ks = torch.tensor(rng.uniform(0.01, 0.05, hkv).astype(np.float32)) if cache == "f8" else None
    vs = torch.tensor(rng.uniform(0.001, 0.05, hkv).astype(np.float32)) if cache == "f8" else None
    fill = torch.tensor(rng.integers(0, 120, (pages, hkv, page, d * ct.itemsize)).astype(np.uint8)).view(ct)
    bufs = []
    for _ in range(2):
        if layout == "tokens":
            x = fill.view(torch.uint8).transpose(1, 2).contiguous().cuda().view(ct).transpose(1, 2)
        else:
            x = fill.clone().cuda()
        bufs.append(x)
    kv = tl.PagedKVCache(pages, page, hkv, d, dtype=ct, k=bufs[0], v=bufs[1], k_scale=None if ks is None else ks.cuda(),
                         v_scale=None if vs is None else vs.cuda())
    out = qd if in_place else None
    got = kv.append(kd, vd, torch.tensor(pos).cuda() if rot else None, torch.tensor(slots).cuda(),
                    cos_sin=torch.tensor(cs).cuda() if rot else None, interleaved=interleaved, q=qd if hq else None, q_out=out)
    assert tl.tl_get_status() == tl.TL_OK

    c, s = cs[pos, :rot // 2], cs[pos, rot // 2:]
    with np.errstate(over="ignore", invalid="ignore"):
        turn = lambda t, w: O.rotate_rows(t.float().numpy(), c, s, rot, interleaved, w)  # noqa: E731
        rq, rk, rv = turn(q, np.float32), turn(k, np.float32), v.float().numpy()
    if hq:
        assert torch.equal(bits(got), bits(torch.tensor(rq).to(dt)))
        ref = turn(q, np.float64)
        ulp = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
        size = np.abs(ref) + 2.0 ** -20 * np.abs(q.double().numpy()).max()
        if spread == 1.0:
            assert np.all(np.abs(got.double().cpu().numpy() - ref) <= ulp * size + 2.0 ** -24)
    else:
        assert got is None
    for rows, scale, buf in ((rk, ks, kv.k), (rv, vs, kv.v)):
        rows = torch.tensor(rows)
        if scale is not None:
            rows = (rows * (1.0 / scale).view(1, -1, 1)).clamp(-448, 448)
        want = fill.view(torch.uint8).clone()
        stored = rows.to(ct).contiguous().view(torch.uint8)
        for t in range(T):
            if slots[t] >= 0:
                want[slots[t] // page, :, slots[t] % page] = stored[t]
        assert torch.equal(buf.contiguous().view(torch.uint8).cpu(), want)       # the other rows are untouched


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f8"), ("f16", "f8")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", [(24, 4, 256, 64), (40, 8, 128, 128), (4, 4, 64, 64), (3, 1, 64, 16), (2, 2, 80, 80),
                                          (5, 1, 96, 32), (1, 1, 512, 512), (4, 2, 128, 0), (0, 2, 128, 128), (33, 1, 16, 16)])
def test_matches_the_formula(dtype, cache, interleaved, hq, hkv, d, rot):
    case(37, hq, hkv, d, 16, dtype, cache, rot, interleaved)


@pytest.mark.parametrize("T", [1, 2, 24, 301, 1300])
@pytest.mark.parametrize("page", [1, 7, 64])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_lengths_pages_and_layouts(T, page, layout):
    case(T, 6, 2, 128, page, layout=layout, seed=T)
    case(T, 6, 2, 128, page, cache="f8", layout=layout, seed=T, interleaved=True, rot=64)


def test_padding_in_place_and_dense_inputs():
    case(40, 6, 2, 128, 16, padded=(0, 7, 39))
    case(40, 6, 2, 128, 16, cache="f8", padded=(3,))
    case(40, 6, 2, 128, 16, in_place=True)
    case(40, 6, 2, 128, 16, in_place=True, interleaved=True, rot=32, dtype="f16")
    case(5, 1, 1, 64, 16, fused=False)


def test_values_beyond_the_stored_type_saturate_or_become_infinite():
    """8 bits saturate at 448 scales; 16 bits round as the type does."""
    case(30, 2, 2, 64, 16, dtype="bf16", cache="f8", spread=100.0)
    case(30, 2, 2, 64, 16, dtype="f16", spread=60000.0 / 4)


def test_nan_and_infinities_pass():
    kv = tl.PagedKVCache(2, 16, 1, 64, dtype=torch.float8_e4m3fn, k_scale=torch.ones(1, device="cuda"), v_scale=torch.ones(1, device="cuda"))
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[0, 0, 3], k[0, 0, 5], k[0, 0, 9] = float("nan"), float("inf"), float("-inf")
    kv.append(k, k, None, torch.tensor([17]).cuda())
    got = kv.v.float().cpu()[1, 0, 1]
    assert torch.isnan(got[3]) and got[5] == 448 and got[9] == -448 and got[0] == 0


def test_bad_positions_and_slots_are_reported():
    kv = tl.PagedKVCache(2, 16, 1, 64)
    k = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    cs = torch.tensor(angles(10, 64)).cuda()
    q = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    hold = torch.full_like(q, 9.0)
    for pos, slots in (([0, 10, 2, 3], [0, 1, 2, 3]), ([0, -1, 2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 32, 2, 3])):
        kv.k.zero_()
        hold.fill_(9.0)
        kv.append(k, k, torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(slots).cuda(), cos_sin=cs, q=q, q_out=hold)
        assert tl.tl_get_status() == tl.TL_EDATA
        live = (kv.k.float().abs().sum(-1) > 0).cpu()[:, 0].reshape(-1)
        assert live.nonzero().flatten().tolist() == [0, 2, 3]
        assert bool((hold[1] == 9).all()) == (pos[1] not in range(10))
        assert bool((hold[0] != 9).all())


def test_cells_past_the_32_bit_range():
    page, hkv, d = 64, 8, 128
    pages = 2 ** 31 // (page * hkv * d) + 40
    k = torch.empty((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    kv = tl.PagedKVCache(pages, page, hkv, d, k=k, v=v)
    x = torch.randn((3, hkv, d), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([pages * page - 1, (pages - 2) * page + 5, 3]).cuda()
    kv.append(x, x * 2, None, slots)
    assert tl.tl_get_status() == tl.TL_OK
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(k[s // page, :, s % page], x[t]) and torch.equal(v[s // page, :, s % page], x[t] * 2)


def test_no_tokens():
    kv = tl.PagedKVCache(2, 16, 2, 64)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert kv.append(e, e, None, torch.empty((0,), dtype=torch.int64, device="cuda")) is None


def test_binding_refusals():
    kv = tl.PagedKVCache(4, 16, 2, 64)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros((3,), dtype=torch.int64, device="cuda")
    cs = torch.zeros((8, 64), device="cuda")
    pos = torch.zeros((3,), dtype=torch.int32, device="cuda")
    for bad in (dict(k=k.float()), dict(v=k[:2]), dict(v=k.half()), dict(k=k.cpu()), dict(slots=slots.int()), dict(slots=slots[:2]),
                dict(positions=pos.long()), dict(cos_sin=cs.double()), dict(q=k[:2]), dict(q=k.half()), dict(q=k, q_out=k[:2])):
        with pytest.raises(ValueError):
            kv.append(**{**dict(k=k, v=k, positions=pos, slots=slots, cos_sin=cs), **bad})
    with pytest.raises(tl.TLError):          # 24 channels cannot be rotated in vectors of 8
        kv.append(k, k, pos, slots, cos_sin=torch.zeros((8, 24), device="cuda"))
    with pytest.raises(tl.TLError):          # the cache's type and the keys' differ
        kv.append(k.half(), k.half(), pos, slots)
    for bad in (dict(dtype=torch.float32), dict(k=kv.k), dict(k_scale=torch.ones(2, device="cuda")), dict(dtype=torch.float8_e4m3fn),
                dict(k=kv.k, v=kv.v[:2]), dict(k=kv.k, v=kv.v.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            tl.PagedKVCache(4, 16, 2, 64, **bad)
