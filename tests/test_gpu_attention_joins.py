"""GPU parity of tl_paged_attention where segments are cut over so many blocks that their partials are joined in two levels,
with other cut segments beside them. Oracle and tolerance are those of test_gpu_paged_attention.py."""

import random

import pytest
import torch

from tests import attention_list as A
from tests.test_gpu_paged_attention import build, check

pytestmark = pytest.mark.gpu


def twice(lens, hq, hkv, d, cache="bf16"):
    """Right twice, and the workspace's counters are zero behind each call."""
    args = build(sum(lens) + hq, lens, hq, hkv, d, 16, cache)
    results = []
    for _ in range(2):
        results.append(check(*args, lens))
        assert not args[0]._ws[:2 * 4096 * 4].any()
    assert torch.equal(*results)
    check(*[args[0], args[1][-1:], args[2][-1:], *args[3:]], lens[-1:])      # another shape through the same workspace


@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([743, 415, 14377, 589], 12, 2, 256), ([122000, 2000], 8, 1, 128), ([157000, 2000], 8, 1, 128), ([2000, 60000, 2000], 16, 1, 128),
    ([90000, 3000, 50000], 32, 1, 128), ([30000, 1, 0, 25000], 6, 1, 256)])
def test_long_and_short_side_by_side(lens, hq, hkv, d):
    twice(lens, hq, hkv, d)


@pytest.mark.parametrize("hq,hkv,d,cache", [(8, 1, 128, "bf16"), (16, 1, 128, "bf16"), (32, 1, 128, "f16"), (12, 2, 256, "bf16"), (8, 1, 256, "f8")])
@pytest.mark.parametrize("blocks_per_sm", [1, 2])
def test_a_lone_last_group_beside_the_next_segment(hq, hkv, d, cache, blocks_per_sm):
    """Lengths for which, on this GPU, the last group of a segment is one partial of the block where the next one begins."""
    blocks = blocks_per_sm * torch.cuda.get_device_properties(0).multi_processor_count
    rng, size, found = random.Random(hq + d), 1 if cache == "f8" else 2, 0
    for _ in range(2000):
        lens = [int(2 ** rng.uniform(8, 16)) for _ in range(rng.randint(2, 5))]
        if A.has_lone_group_beside_a_cut_segment(lens, hkv, hq // hkv, d, size, blocks):
            twice(lens, hq, hkv, d, cache)
            found += 1
            if found == 2:
                return
    assert found > 0


@pytest.mark.parametrize("rest", [0, 1, -1])
def test_every_end_of_the_first_level(rest):
    """One segment of n partials, n - 1 divided by the group's size leaving 0, 1 or the most."""
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    tile = A.tile_keys(128, 2)
    for n in range(90, blocks):
        fan = A.fan_of(n, 8 * 128 * 4)
        if (n - 1) % fan == rest % fan:
            # three places a block; the second segment begins in the first one's last block and takes the rest
            lens = [(3 * n - 3) * tile - 5, 3 * (blocks - n) * tile - 7]
            assert A.cut_segments(lens, 1, tile, blocks) == [(0, 0, 0, n), (1, 0, n - 1, blocks - n + 1)]
            twice(lens, 8, 1, 128)
            return
    assert False
