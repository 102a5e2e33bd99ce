"""How the products of a gated feed-forward block are cut into tiles and parts, on
the host: the library's own header, compiled alone."""
import json
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_mixed_zero1_gb300", "csrc")

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "zero1_gemm_plan.h"
using namespace z1mm;
int main(int, char **argv)
{
    const Plan p = plan_of(atoll(argv[1]), atoll(argv[2]), atoi(argv[3]), 76);
    printf("{\"tn\": %d, \"tiles_m\": %d, \"tiles_n\": %d, \"kblocks\": %d, \"whole\": %d, \"splits\": %d, \"per_split\": %d, "
           "\"bytes\": %lld}", p.tn, p.tiles_m, p.tiles_n, p.kblocks, p.whole, p.splits, p.per_split, (long long)p.bytes);
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


SIZES = [(1, 1, 1), (256, 256, 4), (257, 129, 7), (8192, 28672, 64), (8192, 4096, 448), (14336, 4096, 128), (1, 4096, 448),
         (1, 28672, 64), (300, 200, 2049), (100000, 64, 3), (64, 100000, 17), (5000, 5000, 1)]


@pytest.mark.parametrize("M,N,kblocks", SIZES)
def test_tiles_and_parts_cover_everything_once(plan, M, N, kblocks):
    p = plan(M, N, kblocks)
    assert p["tn"] in (128, 256)
    assert (p["tiles_m"] - 1) * 256 < M <= p["tiles_m"] * 256
    assert (p["tiles_n"] - 1) * p["tn"] < N <= p["tiles_n"] * p["tn"]
    tiles = p["tiles_m"] * p["tiles_n"]
    assert 0 <= p["whole"] <= tiles
    if p["splits"] == 1:
        assert p["whole"] == tiles and p["per_split"] == kblocks
    else:
        assert p["whole"] % 76 == 0 and tiles - p["whole"] < 76 and p["splits"] <= 16
        assert (p["splits"] - 1) * p["per_split"] < kblocks <= p["splits"] * p["per_split"]  # no part is empty
        assert p["per_split"] >= 4


@pytest.mark.parametrize("M,N,kblocks", SIZES)
def test_the_workspace_holds_the_parts(plan, M, N, kblocks):
    p = plan(M, N, kblocks)
    rest = p["tiles_m"] * p["tiles_n"] - p["whole"]
    assert p["bytes"] == (rest * p["splits"] * 256 * p["tn"] * 4 if p["splits"] > 1 else 0)


def test_nothing_to_contract(plan):
    p = plan(300, 500, 0)
    assert p["splits"] == 1 and p["bytes"] == 0
