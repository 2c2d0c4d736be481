"""The plans of prefix attention (CPU): what is chosen from shapes alone, asked of the planning code itself, which a small
program is built with."""
import os
import shutil
import subprocess

import pytest

import test_sanitize as base

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "serve_step.h"
// tokens, sequences, groups, query heads of a cached head, cached heads, d, own keys, prefix keys
int main(int, char** v) {
  int64_t n[8];
  for (int i = 0; i < 8; ++i) n[i] = std::atoll(v[i + 1]);
  wq::PrefixProblem p;
  p.own.N = n[0]; p.own.B = n[1]; p.own.group = n[3]; p.own.hkv = n[4]; p.own.d = n[5]; p.own.page = 16;
  p.shared = p.own;
  p.own.width = n[6] / 16;
  p.shared.B = n[2];
  p.shared.width = n[7] / 16;
  const wq::PrefixPlan pl = wq::plan_prefix(p);
  std::printf("%d %lld %lld %lld %lld\n", (int)pl.split_join, (long long)pl.own.blocks, (long long)pl.own.tiles,
              (long long)pl.shared.blocks, (long long)pl.shared.tiles);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    build = subprocess.run(
        ["g++", "-std=c++17", "-O1", "-I", os.path.join(base.ROOT, "include"), "-I", base.CSRC, str(at / "plan.cpp"),
         os.path.join(base.CSRC, "serve_plan.cpp"), os.path.join(base.CSRC, "serve_step_plan.cpp"), "-o", str(at / "plan")],
        capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    return lambda *n: [int(x) for x in subprocess.run([str(at / "plan"), *map(str, n)], capture_output=True, text=True,
                                                      check=True).stdout.split()]


def test_the_join_is_shared_by_waves_where_tiles_have_many_parts(plan):
    """512 rows of 64 tiles of own keys: few parts of a tile, with short prefixes as without any; long prefixes of few rows
    or few long sequences have many."""
    for groups, keys in ((0, 0), (0, 4096), (8, 64)):
        split, blocks, tiles, shared_blocks, shared_tiles = plan(512, 8, groups, 8, 8, 128, 16384, keys)
        assert blocks < 4 * tiles and (groups == 0) == (shared_tiles == 0)
        assert split == (groups > 0 and shared_blocks >= 4 * shared_tiles), (groups, keys)
    split, blocks, tiles, _, _ = plan(1, 1, 0, 8, 8, 64, 131072, 0)
    assert split and blocks >= 4 * tiles
    split, blocks, tiles, shared_blocks, shared_tiles = plan(64, 64, 1, 4, 8, 128, 1024, 32768)
    assert split and shared_blocks >= 4 * shared_tiles
