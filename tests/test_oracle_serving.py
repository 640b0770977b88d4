"""Pins of the serving oracle (oracle/serving.py) by closed forms and properties, and the serving
entry points' refusals through the C ABI; no GPU."""

import ctypes

import numpy as np
import pytest

from oracle import serving as O
from quantized_linear_layers_block_gb300 import build, tl


@pytest.fixture(scope="module")
def lib():
    build.build()
    return tl.lib()


def angles(pos, rot):
    a = np.asarray(pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    c, s = angles([0, 1, 7, 100, 5000], 32)
    y = O.rotate_rows(x, c, s, 32, interleaved)
    assert np.allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2))
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
    back = O.rotate_rows(y, c, -s, 32, interleaved)
    assert np.allclose(back, x)
    # hand-derived: channel 0 turns by the position itself
    j = 1 if interleaved else 16
    assert np.allclose(y[1, :, 0], x[1, :, 0] * np.cos(1) - x[1, :, j] * np.sin(1))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_products_depend_on_the_distance_only(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    dots = []
    for shift in (0, 5, 1000):
        (cq, sq), (ck, sk) = angles([12 + shift], 64), angles([3 + shift], 64)
        dots.append(np.sum(O.rotate_rows(q, cq, sq, 64, interleaved) * O.rotate_rows(k, ck, sk, 64, interleaved)))
    assert np.allclose(dots, dots[0])


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 6, 2, 4, 8))
    table = np.array([[5, 0, 3], [1, -1, -1], [2, 4, -1]])
    q = rng.standard_normal((3, 4, 8))
    out, lse, _ = O.paged_attention(q, k, v, table, [9, 0, 5], 0.0)
    flat = np.concatenate([v[5], v[0], v[3]], 1)[:, :9]
    assert np.allclose(out[0], np.repeat(flat.mean(1), 2, axis=0))         # scale 0: the mean of the values
    assert np.allclose(lse[0], np.log(9)) and np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))
    out, lse, _ = O.paged_attention(q, k, v, table, [9, 0, 5], 0.3, window=1)
    assert np.allclose(out[2, 0], v[4, 0, 0])                              # one token: its value
    assert np.allclose(lse[2, 3], 0.3 * q[2, 3] @ k[4, 1, 0])


def test_lora_closed_forms():
    rng = np.random.default_rng(3)
    x, base = rng.standard_normal((3, 6)), rng.standard_normal((3, 5))
    A, B = rng.standard_normal((2, 4, 6)), rng.standard_normal((2, 5, 4))
    y, bound = O.lora(x, base, A, B, [2.0, -1.0], [1, -1, 0])
    assert np.array_equal(y[1], base[1])
    assert np.allclose(y[0], base[0] - B[1] @ A[1] @ x[0]) and np.allclose(y[2], base[2] + 2 * (B[0] @ A[0]) @ x[2])
    assert np.all(bound >= np.abs(y - base) - 1e-12)


def _cache(dtype=tl.TL_BF16, **over):
    f = dict(k=4096, v=4096, k_scale=None, v_scale=None, page_stride=2048, head_stride=1024, token_stride=64, dtype=dtype,
             kv_heads=2, head_dim=64, page_size=16, num_pages=4)
    f.update(over)
    return ctypes.pointer(tl.tl_kv_cache(*[f[n] for n, _ in tl.tl_kv_cache._fields_]))


def test_struct_has_the_layout_of_the_header():
    assert ctypes.sizeof(tl.tl_kv_cache) == 4 * 8 + 3 * 8 + 5 * 4 + 4
    assert tl.tl_kv_cache.page_stride.offset == 32 and tl.tl_kv_cache.num_pages.offset == 72


BAD_CACHES = [
    (dict(kv_heads=0), tl.TL_EINVAL), (dict(page_size=0), tl.TL_EINVAL), (dict(num_pages=-1), tl.TL_EINVAL),
    (dict(k=4099), tl.TL_EINVAL), (dict(v=None), tl.TL_EINVAL), (dict(page_stride=0), tl.TL_EINVAL),
    (dict(token_stride=-64), tl.TL_EINVAL), (dict(head_stride=1028), tl.TL_EUNSUPPORTED), (dict(dtype=tl.TL_I8), tl.TL_EINVAL),
    (dict(dtype=tl.TL_F8E4M3), tl.TL_EINVAL), (dict(k_scale=4096, v_scale=4096), tl.TL_EINVAL), (dict(kv_heads=2000), tl.TL_EUNSUPPORTED),
]


def test_append_refusals(lib):
    ok = 4096

    def call(cache=None, q=None, k=ok, v=ok, dtype=tl.TL_BF16, T=3, hq=0, ldq=0, ldk=128, ldv=128, qo=None, ldo=0, cs=None, mp=0, rot=0,
             il=0, pos=None, slots=ok):
        return lib.tl_kv_append(cache or _cache(), q, k, v, dtype, T, hq, ldq, ldk, ldv, qo, ldo, cs, mp, rot, il, pos, slots, None)

    for over, code in BAD_CACHES:
        assert call(cache=_cache(**over)) == code, over
    assert lib.tl_kv_append(None, None, ok, ok, tl.TL_BF16, 0, 0, 0, 0, 0, None, 0, None, 0, 0, 0, None, None, None) == tl.TL_EINVAL
    assert call(dtype=tl.TL_F32) == tl.TL_EINVAL
    assert call(dtype=tl.TL_F16) == tl.TL_EINVAL             # the cache is bf16
    assert call(T=-1) == tl.TL_EINVAL
    assert call(k=None) == tl.TL_EINVAL
    assert call(slots=None) == tl.TL_EINVAL
    assert call(slots=4100) == tl.TL_EINVAL
    assert call(v=4096 + 8) == tl.TL_EINVAL
    assert call(il=2) == tl.TL_EINVAL
    assert call(rot=16, mp=5) == tl.TL_EINVAL                # no table
    assert call(rot=16, mp=5, cs=ok) == tl.TL_EINVAL         # no positions
    assert call(rot=24, mp=5, cs=ok, pos=ok) == tl.TL_EUNSUPPORTED
    assert call(rot=80, mp=5, cs=ok, pos=ok) == tl.TL_EUNSUPPORTED
    assert call(cache=_cache(head_dim=24)) == tl.TL_EUNSUPPORTED
    assert call(cache=_cache(head_dim=528)) == tl.TL_EUNSUPPORTED
    assert call(ldk=132) == tl.TL_EUNSUPPORTED
    assert call(ldk=64) == tl.TL_EUNSUPPORTED                # tokens overlap
    assert call(ldv=-128) == tl.TL_EINVAL
    assert call(q=ok, hq=4, ldq=256, qo=None) == tl.TL_EINVAL
    assert call(q=ok, hq=4, ldq=250, qo=ok, ldo=256) == tl.TL_EUNSUPPORTED
    assert call(q=ok, hq=4, ldq=256, qo=ok, ldo=264) == tl.TL_EINVAL      # in place, but the rows lie elsewhere
    assert call(T=0, k=None, v=None, slots=None) == tl.TL_OK


def test_attention_refusals(lib):
    ok = 4096

    def call(cache=None, q=ok, dtype=tl.TL_BF16, B=3, hq=4, ldq=256, pages=ok, mp=2, ldp=2, lens=ok, scale=0.1, window=0, out=ok, ldo=256,
             lse=None, ws=ok, wsb=0):
        return lib.tl_paged_attention(cache or _cache(), q, dtype, B, hq, ldq, pages, mp, ldp, lens, scale, window, out, ldo, lse, ws, wsb,
                                      None)

    for over, code in BAD_CACHES:
        assert call(cache=_cache(**over)) == code, over
    assert call(dtype=tl.TL_F32) == tl.TL_EINVAL
    assert call(dtype=tl.TL_F16) == tl.TL_EINVAL
    assert call(cache=_cache(head_dim=96)) == tl.TL_EUNSUPPORTED
    assert call(hq=5) == tl.TL_EUNSUPPORTED
    assert call(hq=258) == tl.TL_EUNSUPPORTED                # 129 query heads on one key-value head
    assert call(hq=0) == tl.TL_EINVAL
    assert call(B=-1) == tl.TL_EINVAL
    assert call(window=-1) == tl.TL_EINVAL
    assert call(scale=float("nan")) == tl.TL_EINVAL
    assert call(scale=float("inf")) == tl.TL_EINVAL
    for name in ("q", "out", "lens", "pages", "ws"):
        assert call(**{name: None}) == tl.TL_EINVAL, name
    assert call(q=4104) == tl.TL_EINVAL
    assert call(lens=4098) == tl.TL_EINVAL
    assert call(ldp=1) == tl.TL_EINVAL
    assert call(ldq=252) == tl.TL_EUNSUPPORTED
    assert call(ldo=128) == tl.TL_EUNSUPPORTED
    assert call(B=0, q=None, out=None, lens=None, pages=None, ws=None) == tl.TL_OK
    sz = ctypes.c_size_t(9)
    assert lib.tl_paged_attention_workspace_size(0, 4, 2, 64, ctypes.byref(sz)) == tl.TL_OK and sz.value == 0
    assert lib.tl_paged_attention_workspace_size(1, 4, 3, 64, ctypes.byref(sz)) == tl.TL_EUNSUPPORTED
    assert lib.tl_paged_attention_workspace_size(1, 4, 2, 64, None) == tl.TL_EINVAL


def test_division_by_multiplication():
    """The page of a token: n / d as (n m) >> (31 + s), exact for n < 2^31."""
    rng = np.random.default_rng(4)
    for d in [1, 2, 3, 7, 16, 24, 100, 256, 1000, 65535, 2 ** 20 + 1, 2 ** 30 - 1, 2 ** 30 + 1, 2 ** 31 - 1]:
        s = max(0, (d - 1).bit_length())
        m = 2 ** (31 + s) // d + 1
        assert m < 2 ** 32
        ns = [0, 1, d - 1, d, d + 1, 2 * d - 1, 2 ** 31 - 1] + [int(x) for x in rng.integers(0, 2 ** 31, 200)]
        ns += [k * d + e for k in (2 ** 31 // d - 1, 2 ** 31 // d // 2) for e in (-1, 0)]
        for n in ns:
            if 0 <= n < 2 ** 31:
                assert (n * m) >> (31 + s) == n // d, (n, d)


def test_lora_refusals(lib):
    ok = 4096

    def call(x=ok, ldx=64, A=ok, B=ok, scale=ok, dtype=tl.TL_BF16, n=2, rank=16, plan=ok, M=3, N=128, K=64, base=ok, ldb=128, y=8192, ldy=128,
             yd=tl.TL_BF16):
        return lib.tl_lora_apply(x, ldx, A, B, scale, dtype, n, rank, plan, M, N, K, base, ldb, y, ldy, yd, None)

    for name in ("x", "A", "B", "scale", "plan", "base", "y"):
        assert call(**{name: None}) == tl.TL_EINVAL, name
        assert call(**{name: 4098}) == tl.TL_EINVAL, name
    assert call(dtype=tl.TL_F32) == tl.TL_EINVAL
    assert call(yd=tl.TL_F8E4M3) == tl.TL_EINVAL
    assert call(M=-1) == tl.TL_EINVAL
    assert call(K=0) == tl.TL_EINVAL
    for over in (dict(rank=12), dict(rank=136), dict(K=60), dict(N=100), dict(ldx=56), dict(ldy=132), dict(n=9000), dict(M=(1 << 20) + 1),
                 dict(N=(1 << 22) + 8)):
        assert call(**over) == tl.TL_EUNSUPPORTED, over
    assert call(y=ok, ldy=136) == tl.TL_EINVAL               # in place, but the rows lie elsewhere
    assert call(M=0, x=None, base=None, y=None, plan=None) == tl.TL_OK
    assert call(N=0, x=None, base=None, y=None, plan=None) == tl.TL_OK
    sz = ctypes.c_size_t()
    assert lib.tl_lora_plan_size(33, 4, ctypes.byref(sz)) == tl.TL_OK and sz.value == 16 + 144 * (1 + 5)
    assert lib.tl_lora_plan_size(2, 400, ctypes.byref(sz)) == tl.TL_OK and sz.value == 16 + 144 * 2
    assert lib.tl_lora_plan(None, 2, 4, ok, 10 ** 6, None) == tl.TL_EINVAL
    assert lib.tl_lora_plan(ok, 2, 4, ok, 10, None) == tl.TL_ENOSPACE
    assert lib.tl_lora_plan(ok, 2, 9000, ok, 10 ** 9, None) == tl.TL_EUNSUPPORTED
    assert lib.tl_lora_plan(None, 0, 4, None, 0, None) == tl.TL_OK
