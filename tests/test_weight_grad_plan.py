"""How a weight gradient is cut into tiles, parts and joining launches, on the
host: the library's own header, compiled alone."""
import json
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_mixed_zero1_gb300", "csrc")

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "zero1_weight_grad_plan.h"
using namespace z1wg;
int main(int argc, char **argv)
{
    if (argc == 2) {  // every state that a use of B's place can be left in
        printf("[");
        for (unsigned mine = 0; mine < 2; ++mine)
            for (unsigned other = 0; other < 2; ++other)
                for (unsigned late = 0; late <= 8; ++late) {
                    const Drain d = drain_of(5, 5 + mine, 5 + other, late);
                    printf("%s[%u, %u, %u, %u, %u, %u]", mine + other + late ? ", " : "", mine, other, late, d.arrivals,
                           d.announce, d.write_off);
                }
        printf("]");
        return 0;
    }
    const long tiles_k = atol(argv[1]), tiles_n = atol(argv[2]), kblocks = atol(argv[3]), limit = atol(argv[4]);
    Plan p{};
    p.tiles_k = (int)tiles_k; p.tiles_n = (int)tiles_n; p.kblocks = (int)kblocks; p.clusters = 76;
    split_rest(&p);
    printf("{\"tiles\": %ld, \"whole\": %d, \"splits\": %d, \"per_split\": %d, \"runs\": [", tiles_k * tiles_n, p.whole,
           p.splits, p.per_split);
    for (int t = p.whole, tiles = p.tiles_k * p.tiles_n; t < tiles;) {
        const JoinRun r = join_run(p.whole, tiles, p.splits, t, (int)limit);
        printf("%s[%d, %d, %lld]", t == p.whole ? "" : ", ", r.tile, r.tiles, (long long)r.part);
        t += r.tiles;
    }
    printf("]}");
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, exe = str(d / "plan.cpp"), str(d / "plan")
    with open(src, "w") as f:
        f.write(DRIVER)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-Wall", "-Werror", "-I", CSRC, src, "-o", exe], check=True)
    return lambda *a: json.loads(subprocess.run([exe, *map(str, a)], check=True, capture_output=True).stdout)


CASES = [(16, 16, 128), (16, 56, 128), (4, 4, 13), (5, 1, 2049), (257, 257, 2050), (20, 31, 2100), (1, 1, 1)]


@pytest.mark.parametrize("tiles_k,tiles_n,kblocks", CASES)
def test_parts_cover_the_rows(plan, tiles_k, tiles_n, kblocks):
    p = plan(tiles_k, tiles_n, kblocks, 65535)
    assert 1 <= p["splits"] <= 16 and 0 <= p["whole"] <= p["tiles"]
    assert (p["splits"] - 1) * p["per_split"] < kblocks <= p["splits"] * p["per_split"]   # no part is empty
    if kblocks > 2048:
        assert p["whole"] == 0 and p["splits"] > 1    # a whole tile's rows fit one run of the accumulator


@pytest.mark.parametrize("tiles_k,tiles_n,kblocks", CASES)
@pytest.mark.parametrize("limit", [1, 7, 65535])
def test_each_joined_tile_gets_its_own_parts(plan, tiles_k, tiles_n, kblocks, limit):
    """Whatever the launches' size, tile t's parts are those that the main
    kernel wrote for it: (t - whole) * splits tiles of 256 x 256 values in."""
    p = plan(tiles_k, tiles_n, kblocks, limit)
    seen = {}
    for first, count, part in p["runs"]:
        assert 1 <= count <= limit
        for k in range(count):
            assert first + k not in seen
            seen[first + k] = part + k * p["splits"] * 65536          # what block k of the launch reads
    assert sorted(seen) == list(range(p["whole"], p["tiles"]))
    assert all(at == (t - p["whole"]) * p["splits"] * 65536 for t, at in seen.items())


def test_what_is_made_up_waits_for_the_loads_under_way(plan):
    """A barrier of nine arrivals and two halves of bytes (the leading CTA's load
    announces both and is one arrival; eight converting warps) after the pair has
    given up: the use becomes complete exactly when every half that was loaded
    has landed, whenever that is, and no half lands on a completed use."""
    states = plan("drain")
    assert len(states) == 36
    for mine, other, late, arrivals, announce, write_off in states:
        if not mine and not other:
            continue                                       # past the last use: not asked for
        for before in range(mine + other + 1):             # halves that land before the barrier is made up
            pending, bytes_due = 9 - mine - (8 - late), 2 * mine - before
            done = pending == 0 and bytes_due == 0
            assert not done or (before == mine + other and not (arrivals or announce or write_off))
            under_way = mine + other - before
            bytes_due += announce
            bytes_due -= write_off
            assert arrivals <= pending                     # never one arrival too many
            assert not (pending == 0 and bytes_due == 0 and under_way)
            pending -= arrivals
            assert pending == 0
            while under_way:
                assert bytes_due != 0                      # not complete yet
                bytes_due, under_way = bytes_due - 1, under_way - 1
            assert bytes_due == 0
