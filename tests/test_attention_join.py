"""The counters by which blocks of paged attention find out who joins a segment's partials: no counter has two users,
every partial reaches exactly one join on each level, and all lies inside the workspace; no GPU."""

import random

import pytest

from tests import attention_list as A


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    return A.JoinRule(str(tmp_path_factory.mktemp("join")))


def users(rule, cut, heads, dim):
    """{counter: (request, head group, level, first)}; fails where a counter gets a second user."""
    seen = {}
    for b, h, c0, n in cut:
        fan = rule.fan(n, heads * dim * 4)
        assert fan == A.fan_of(n, heads * dim * 4) and (fan == n or fan * fan >= n) and fan >= 2
        blocks, step, level = list(range(n)), 1, 0
        while len(blocks) > 1:
            groups = {}
            for i in blocks:
                first, size, counter = rule.group(c0 + i, c0, n, fan, step, level)
                groups.setdefault(first, []).append(i)
                assert first % (step * fan) == 0 and (counter < 0) == (size == 1)
                if counter >= 0:
                    assert counter < rule.counters
                    mine = (b, h, level, first)
                    assert seen.setdefault(counter, mine) == mine, (counter, seen[counter], mine)
            for first, members in groups.items():
                assert members[0] == first and len(members) == rule.group(c0 + first, c0, n, fan, step, level)[1]
            blocks, step, level = sorted(groups), step * fan, level + 1
        assert blocks == [0]
    return seen


@pytest.mark.parametrize("lens,head_groups,heads,dim,blocks", [
    ([743, 415, 14377, 589], 2, 6, 256, 152), ([122000, 2000], 1, 8, 128, 304), ([157000, 2000], 1, 8, 128, 304)])
def test_a_lone_last_group_beside_the_next_segment(rule, lens, head_groups, heads, dim, blocks):
    assert A.has_lone_group_beside_a_cut_segment(lens, head_groups, heads, dim, 2, blocks)
    users(rule, A.cut_segments(lens, head_groups, A.tile_keys(dim, 2), blocks), heads, dim)


def test_random_batches(rule):
    rng = random.Random(0)
    lone = 0
    for _ in range(3000):
        dim, heads, size = rng.choice([(64, 8, 2), (128, 8, 1), (128, 16, 2), (128, 32, 2), (256, 6, 2), (256, 16, 1), (256, 16, 2)])
        lens = [int(2 ** rng.uniform(0, 17)) for _ in range(rng.randint(1, 12))]
        groups, blocks = rng.choice([1, 1, 2, 3, 4]), rng.choice([152, 304, 148, 296])
        users(rule, A.cut_segments(lens, groups, A.tile_keys(dim, size), blocks), heads, dim)
        lone += A.has_lone_group_beside_a_cut_segment(lens, groups, heads, dim, size, blocks)
    assert lone >= 10            # the case that needs it does come up


def test_every_number_of_blocks(rule):
    for n in range(2, 305):
        for heads, dim in ((1, 64), (8, 128), (6, 256), (16, 256), (32, 128)):
            users(rule, [(0, 0, 0, n), (1, 0, n - 1, 9)], heads, dim)
