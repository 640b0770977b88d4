"""tl_paged_attention over values that are infinite or NaN: sum_j p_j V_j of each channel by the arithmetic of infinities, all
else bit for bit what it is without them."""

import numpy as np
import pytest
import torch

from quantized_linear_layers_block_gb300 import tl
from tests.test_gpu_paged_attention import build, check

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# what stands in a channel's values of a few keys, and the channel's result
PLANTED = [((INF,), INF), ((-INF,), -INF), ((INF, INF, INF), INF), ((INF, -INF), NAN), ((NAN,), NAN), ((INF, NAN), NAN), ((-INF, -INF), -INF)]

# (lens, query heads, key-value heads, window) of each form of the kernel: clusters, single rings, the list with segments cut
# over blocks, a window
FORMS = {
    "cluster": ([700, 40], 6, 2, 0),
    "fours": ([600, 450] * 7, 16, 4, 0),
    "twos": ([600, 450] * 19, 12, 4, 0),
    "block": ([50] * 40, 4, 2, 0),
    "rings": ([30, 1, 9, 60] * 120, 4, 2, 0),
    "list": ([9000, 33, 5000, 700], 10, 2, 0),
    "many heads": ([3000, 20, 900], 33, 1, 0),
    "window": ([900, 300, 70], 12, 1, 100),
}


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("form", list(FORMS))
def test_infinite_and_nan_values(form, d, cache):
    lens, hq, hkv, window = FORMS[form]
    kv, q, table, k64, v64 = build(d + hq, lens, hq, hkv, d, 16, cache)
    good = check(kv, q, table, k64, v64, lens, window=window)
    rng = np.random.default_rng(d)
    td, ld, group = torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), hq // hkv
    want = good.clone()
    for i, (values, result) in enumerate(PLANTED):
        b, h, c = 2 * i % len(lens), i % hkv, 1 + 3 * i
        n = lens[b]
        first = max(0, n - window) if window else 0
        if n - first < len(values):
            continue
        for j, x in zip(rng.choice(np.arange(first, n), len(values), replace=False), values):
            kv.v[table[b, j // 16], h, j % 16, c] = x
        want[b, h * group:(h + 1) * group, c] = result
    lse = torch.empty((len(lens), hq), device="cuda")
    y = kv.attend(q.cuda(), td, ld, window=window, lse=lse)
    assert tl.tl_get_status() == tl.TL_OK
    assert not torch.isfinite(want).all() and bool(torch.isfinite(lse).all())
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y, nan=0.0, posinf=1e4, neginf=-1e4), torch.nan_to_num(want, nan=0.0, posinf=1e4, neginf=-1e4))


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("form", list(FORMS))
def test_infinite_values_of_keys_without_weight(form, cache):
    """p_j is positive however far a key's score lies below the others': e^-1000 of an infinity is one."""
    lens, hq, hkv, window = FORMS[form]
    kv, q, table, _, _ = build(3, lens, hq, hkv, 128, 16, cache)
    td, ld, group = torch.tensor(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), hq // hkv
    args = dict(scale=200.0, window=window)      # scores some thousand apart
    want = kv.attend(q.cuda(), td, ld, **args).clone()
    assert bool(torch.isfinite(want).all())
    rng = np.random.default_rng(4)
    for b in range(0, len(lens), 3):
        n = lens[b]
        first = max(0, n - window) if window else 0
        for c in range(8):
            j, x, h = rng.integers(first, n), (INF, -INF)[c % 2], int(rng.integers(hkv))
            kv.v[table[b, j // 16], h, j % 16, 5 * c + 1] = x
            want[b, h * group:(h + 1) * group, 5 * c + 1] = x
    assert torch.equal(kv.attend(q.cuda(), td, ld, **args), want)


def test_infinite_keys():
    """A score of +inf or NaN makes all of its head NaN; one of -inf is a key without weight."""
    lens = [40, 40]
    kv, q, table, k64, v64 = build(17, lens, 2, 1, 64, 16, "f16")
    q = torch.ones_like(q)
    good = check(kv, q, table, k64, v64, lens)
    lens_d, table_d = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(table).cuda()
    keep = kv.k[table[0, 1], 0, 3].clone()
    kv.k[table[0, 1], 0, 3, 5] = INF
    y = kv.attend(q.cuda(), table_d, lens_d)
    assert bool(torch.isnan(y[0]).all()) and torch.equal(y[1], good[1])
    kv.k[table[0, 1], 0, 3, 5] = -INF
    y = kv.attend(q.cuda(), table_d, lens_d)
    kv.k[table[0, 1], 0, 3] = keep
    k64 = k64.copy()
    k64[table[0, 1], 0, 3, 5] = -1e30           # the same without an infinity in the oracle's arithmetic
    kv.k[table[0, 1], 0, 3, 5] = -6e4
    assert torch.equal(y[0], kv.attend(q.cuda(), table_d, lens_d)[0]) and torch.equal(y[1], good[1])
