"""The entry points for drafted trees refuse what include/tl.h says they refuse, before any CUDA call; no GPU."""

import ctypes

import pytest
import torch

from quantized_linear_layers_block_gb300 import build, tl
from tests.test_devices import BF, F, I, L, U8, arguments, fake, refused, tensors

OK, EINVAL, EUNSUPPORTED = tl.TL_OK, tl.TL_EINVAL, tl.TL_EUNSUPPORTED
P = ctypes.c_void_p
ok, off4, off8, off16 = P(4096), P(4096 + 2), P(4096 + 4), P(4096 + 8)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return tl.lib()


def cache(**change):
    c = tl.tl_kv_cache(k=4096, v=4096, page_stride=2 * 16 * 64, head_stride=16 * 64, token_stride=64, dtype=tl.TL_BF16, kv_heads=2, head_dim=64,
                       page_size=16, num_pages=4)
    for k, v in change.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def call(f, defaults, **change):
    assert set(change) <= set(defaults), change
    return f(*{**defaults, **change}.values())


def test_plan(lib):
    d = dict(parents=ok, starts=ok, B=2, T=6, lens=ok, pages=ok, max_pages=3, ldp=3, page_size=16, num_pages=4, masks=ok, positions=ok, slots=ok, stream=None)
    for bad in (dict(B=-1), dict(T=-1), dict(max_pages=-1), dict(page_size=0), dict(num_pages=-1), dict(parents=None), dict(starts=None), dict(lens=None),
                dict(pages=None), dict(masks=None), dict(positions=None), dict(slots=None), dict(ldp=2), dict(parents=off4), dict(starts=off4),
                dict(lens=off4), dict(pages=off4), dict(positions=off4), dict(masks=off8), dict(slots=off8)):
        assert call(lib.tl_tree_plan, d, **bad) == EINVAL, bad
    assert call(lib.tl_tree_plan, d, B=0, T=0, starts=None, lens=None, pages=None, parents=None, masks=None, positions=None, slots=None) == OK
    assert call(lib.tl_tree_plan, d, T=0) == OK


def test_attention(lib):
    d = dict(cache=cache(), q=ok, dtype=tl.TL_BF16, B=2, T=6, q_heads=4, ldq=256, masks=ok, starts=ok, pages=ok, max_pages=3, ldp=3, lens=ok, scale=0.1,
             window=0, sinks=0, out=ok, ldo=256, lse=None, workspace=ok, ws_bytes=1 << 40, stream=None)
    f = lib.tl_tree_attention
    for bad in (dict(q=None), dict(out=None), dict(masks=None), dict(starts=None), dict(pages=None), dict(lens=None), dict(workspace=None), dict(B=-1), dict(T=-1),
                dict(q_heads=0), dict(dtype=tl.TL_F32), dict(dtype=tl.TL_F16), dict(window=-1), dict(sinks=-1), dict(sinks=4), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=off16), dict(out=off16), dict(workspace=off16), dict(masks=off8), dict(starts=off4), dict(lens=off4),
                dict(pages=off4), dict(lse=off4), dict(ldp=2), dict(max_pages=-1), dict(ldq=-8), dict(cache=cache(page_size=0)), dict(cache=None)):
        assert call(f, d, **bad) == EINVAL, bad
    for bad in (dict(window=63), dict(window=1), dict(q_heads=5), dict(q_heads=2 * 129), dict(cache=cache(head_dim=32)), dict(cache=cache(head_dim=512)),
                dict(ldq=252), dict(ldq=248), dict(ldo=250), dict(cache=cache(token_stride=68))):
        assert call(f, d, **bad) == EUNSUPPORTED, bad
    assert call(f, d, B=0, T=0, q=None) == OK and call(f, d, T=0) == OK
    n = ctypes.c_size_t(7)
    size = lib.tl_tree_attention_workspace_size
    assert size(0, 0, 4, 2, 64, ctypes.byref(n)) == OK and n.value == 0
    assert size(1, 1, 4, 2, 96, ctypes.byref(n)) == EUNSUPPORTED and size(-1, 1, 4, 2, 64, ctypes.byref(n)) == EINVAL
    assert size(1, -1, 4, 2, 64, ctypes.byref(n)) == EINVAL and size(1, 1, 4, 2, 64, None) == EINVAL


def test_verify(lib):
    d = dict(target=ok, ldt=100, draft=ok, ldd=100, vocab=100, tokens=ok, parents=ok, starts=ok, B=2, T=6, uniform=ok, path=ok, counts=ok, next=ok, stream=None)
    f = lib.tl_verify_tree
    for bad in (dict(target=None), dict(tokens=None), dict(parents=None), dict(starts=None), dict(uniform=None), dict(path=None), dict(counts=None),
                dict(next=None), dict(B=-1), dict(T=-1), dict(vocab=0), dict(vocab=-5), dict(ldt=-1), dict(target=off4), dict(draft=off4), dict(tokens=off4),
                dict(path=off4)):
        assert call(f, d, **bad) == EINVAL, bad
    for bad in (dict(vocab=(1 << 24) + 1, ldt=1 << 25, ldd=1 << 25), dict(ldt=99), dict(ldd=99)):
        assert call(f, d, **bad) == EUNSUPPORTED, bad
    assert call(f, d, B=0, T=0) == OK


def test_compact(lib):
    d = dict(cache=cache(), path=ok, counts=ok, starts=ok, B=2, T=6, pages=ok, max_pages=3, ldp=3, lens=ok, stream=None)
    f = lib.tl_kv_compact
    for bad in (dict(path=None), dict(counts=None), dict(starts=None), dict(pages=None), dict(lens=None), dict(B=-1), dict(T=-1), dict(max_pages=-1),
                dict(ldp=1), dict(path=off4), dict(counts=off4), dict(cache=None), dict(cache=cache(kv_heads=0))):
        assert call(f, d, **bad) == EINVAL, bad
    for bad in (dict(cache=cache(head_dim=24)), dict(cache=cache(head_dim=528)), dict(cache=cache(page_stride=12))):
        assert call(f, d, **bad) == EUNSUPPORTED, bad
    assert call(f, d, B=0) == OK and call(f, d, T=0) == OK


def test_append_norm(lib):
    d = dict(cache=cache(), q=ok, k=ok, v=ok, dtype=tl.TL_BF16, T=3, q_heads=4, ldq=256, ldk=128, ldv=128, q_out=ok, ldqo=256, q_norm=ok, k_norm=ok, eps=1e-6,
             cos_sin=ok, max_pos=8, rot_dim=64, interleaved=0, positions=ok, slots=ok, stream=None)
    f = lib.tl_kv_append_norm
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(q_norm=off16), dict(k_norm=off16), dict(k=None),
                dict(q_out=None), dict(slots=None), dict(dtype=tl.TL_F16), dict(interleaved=2)):
        assert call(f, d, **bad) == EINVAL, bad
    assert call(f, d, rot_dim=24) == EUNSUPPORTED and call(f, d, T=0) == OK


@pytest.fixture(scope="module")
def mod(lib):
    return tl._tensors()


def test_module_arguments(mod):
    for f in (mod.kv_append_norm, mod.tree_plan, mod.tree_attention, mod.verify_tree, mod.kv_compact):
        for n in (0, 30):
            with pytest.raises(TypeError):
                f(*[None] * n)
    x = torch.zeros(2, 2, 64)
    for bad in (x, None, 3):
        for f, n in ((mod.tree_plan, 9), (mod.tree_attention, 13), (mod.kv_compact, 7), (mod.kv_append_norm, 13)):
            with pytest.raises(ValueError):
                f(0, bad, *[x] * (n - 2))
        with pytest.raises(ValueError):
            mod.verify_tree(bad, *[x] * 9)


two = pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2, reason="one GPU: tensors of another cannot be named")
PLAN = [("parents", (6,), I), ("starts", (4,), I), ("lens", (3,), I), ("pages", (3, 2), I), ("masks", (6,), L), ("positions", (6,), I), ("slots", (6,), L),
        ("stream", None, None)]
TREE = [("q", (6, 4, 64), BF), ("masks", (6,), L), ("starts", (4,), I), ("pages", (3, 2), I), ("lens", (3,), I), ("scale", None, 1.0), ("window", None, 0),
        ("sinks", None, 0), ("out", (6, 4, 64), BF), ("lse", (6, 4), F), ("workspace", (64,), U8), ("stream", None, None)]
VERIFY = [("target", (6, 100), F), ("draft", (6, 100), F), ("tokens", (6,), I), ("parents", (6,), I), ("starts", (4,), I), ("uniform", (6,), F),
          ("path", (6,), I), ("counts", (3,), I), ("next", (3,), I), ("stream", None, None)]
COMPACT = [("path", (6,), I), ("counts", (3,), I), ("starts", (4,), I), ("pages", (3, 2), I), ("lens", (3,), I), ("stream", None, None)]
ON_CACHE = {"tree_plan": PLAN, "tree_attention": TREE, "kv_compact": COMPACT}


def bound(device=0):
    return tl._Cache(tl.tl_kv_cache(dtype=tl.TL_BF16, kv_heads=2, head_dim=64, page_size=16, num_pages=4), device)


@two
@pytest.mark.parametrize("f,away", [(f, name) for f, spec in ON_CACHE.items() for name in tensors(spec)])
def test_tensors_of_another_gpu(mod, f, away):
    c = bound()
    refused(getattr(mod, f), ctypes.addressof(c), *arguments(ON_CACHE[f], away))


@two
@pytest.mark.parametrize("away", tensors(VERIFY))
def test_verify_tensors_of_another_gpu(mod, away):
    if away == "target":           # the call is where the target is
        away = "draft"
    refused(mod.verify_tree, *arguments(VERIFY, away))


@two
@pytest.mark.parametrize("f", list(ON_CACHE))
def test_cache_on_another_gpu(mod, f):
    c = bound(1)
    refused(getattr(mod, f), ctypes.addressof(c), *arguments(ON_CACHE[f], None))


@two
@pytest.mark.parametrize("f,name,shape,dtype", [
    ("tree_plan", "starts", (4, 1), I), ("tree_plan", "starts", (0,), I), ("tree_plan", "lens", (4,), I), ("tree_plan", "pages", (2, 2), I),
    ("tree_plan", "masks", (6,), I), ("tree_plan", "slots", (5,), L), ("tree_plan", "parents", (6,), L), ("tree_attention", "q", (6, 4, 32), BF),
    ("tree_attention", "q", (6, 4, 64), F), ("tree_attention", "masks", (7,), L), ("tree_attention", "out", (5, 4, 64), BF), ("tree_attention", "lse", (6, 5), F),
    ("kv_compact", "counts", (2,), I), ("kv_compact", "path", (6,), L)])
def test_shapes_and_types(mod, f, name, shape, dtype):
    spec = [(n, shape, dtype) if n == name else (n, s, d) for n, s, d in ON_CACHE[f]]
    c = bound()
    with pytest.raises(ValueError):
        getattr(mod, f)(ctypes.addressof(c), *arguments(spec, None))


@two
@pytest.mark.parametrize("name,shape,dtype", [("target", (6, 100), BF), ("draft", (6, 99), F), ("tokens", (5,), I), ("uniform", (6,), I), ("counts", (4,), I),
                                              ("starts", (4,), L)])
def test_verify_shapes_and_types(mod, name, shape, dtype):
    with pytest.raises(ValueError):
        mod.verify_tree(*arguments([(n, shape, dtype) if n == name else (n, s, d) for n, s, d in VERIFY], None))


def test_tree_oracle():
    """The oracle's masks, what a node sees, and that its verification is the textbook's on a chain."""
    import numpy as np
    from oracle import serving as O
    assert O.tree_masks([-1, 0, 0, 1, 3, -1]) == [1, 3, 5, 11, 27, 32]
    assert O.tree_seen(5, 0b1011) == [0, 1, 2, 3, 4, 5, 6, 8]
    assert O.tree_seen(10, 0b11, window=4, sinks=1) == [0, 8, 9, 10, 11] and O.tree_seen(10, 0b11111, window=4, sinks=0) == [10, 11, 12, 13, 14]
    p, q = np.array([[.5, .3, .2]] * 2), np.array([[.2, .3, .5]] * 2)
    for u, want in ((.39, [0, 1]), (.41, [0])):                  # accepted with probability p / q = 0.4
        assert O.verify_tree(p, q, [0, 2], [-1, 0], [0.0, u])[0] == want
    assert O.verify_tree(p, q, [0, 2], [-1, 0], [0.99, .41]) == ([0], 0)      # the rest is all on token 0
    assert np.allclose(O.head_norm(np.full((1, 1, 4), 3.0), np.ones(4), 0), 1)
