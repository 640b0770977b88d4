"""How paged attention cuts its list of key tiles into the blocks' shares, restated; and the library's own rule of who
joins the partials of a segment (csrc/attention_join.h), compiled for the CPU."""

import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_linear_layers_block_gb300", "csrc")

SHIM = """
#include "attention_join.h"
extern "C" int fan(int n, int bytes) { return tl::attn::join_fan(n, bytes); }
extern "C" void group(int block, int c0, int n, int fan, int step, int level, int* out) {
  const tl::attn::JoinGroup g = tl::attn::join_group(block, c0, n, fan, step, level);
  out[0] = g.first, out[1] = g.size, out[2] = g.counter;
}
extern "C" int counters() { return tl::kAttnLevels * tl::kAttnMaxGrid; }
"""


class JoinRule:
    def __init__(self, folder):
        src, lib = os.path.join(folder, "join.cpp"), os.path.join(folder, "join.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)
        self.fan = self.lib.fan
        self.counters = self.lib.counters()

    def group(self, block, c0, n, fan, step, level):
        out = (ctypes.c_int * 3)()
        self.lib.group(block, c0, n, fan, step, level, out)
        return tuple(out)


def tile_keys(dim, cache_bytes):
    """Keys of a tile of the whole block: four rings of 4 KB of K each, at least 16 keys."""
    return 4 * max(16, 4096 // (dim * cache_bytes))


def cut_segments(lens, head_groups, tile, blocks):
    """[(request, group of heads, c0, n)] of the segments that n >= 2 blocks share, from block c0 on.

    The list: for each request and group of heads one place for what a segment costs besides its tiles, then its tiles;
    each block takes an equal share of the places.
    """
    tiles = [max(1, -(-n // tile)) for n in lens]
    total = head_groups * sum(t + 1 for t in tiles)
    share = -(-total // min(blocks, total))
    cut, at = [], 0
    for b, t in enumerate(tiles):
        for h in range(head_groups):
            first = at + 1
            c0, c1 = first // share, (first + t - 1) // share
            if c1 > c0:
                cut.append((b, h, c0, c1 - c0 + 1))
            at += t + 1
    return cut


def fan_of(n, partial_bytes):
    """Partials to a group, as the rule above has it."""
    return n if n * partial_bytes <= 320 * 1024 else next(f for f in range(1, n + 1) if f * f >= n)


def has_lone_group_beside_a_cut_segment(lens, head_groups, heads, dim, cache_bytes, blocks):
    """Whether the last group of some segment is one partial, of the block in which the next cut segment begins."""
    cut = cut_segments(lens, head_groups, tile_keys(dim, cache_bytes), blocks)
    starts = {c0 for _, _, c0, _ in cut}
    return any((n - 1) % fan_of(n, heads * dim * 4) == 0 and c0 + n - 1 in starts for _, _, c0, n in cut if fan_of(n, heads * dim * 4) < n)
