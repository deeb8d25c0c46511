"""The kernel's own cuts (csrc/pa_split_plan.h) driven on the CPU: the header is compiled as plain C++ and agrees with
the restatement, which test_split_plan.py checks, on random batches and on every unit of small ones."""
import os
import random
import shutil
import subprocess

import pytest

from test_split_plan import place, shares

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_149_gb300", "csrc")

# a batch per line: cut, grid, total, then n and n numbers (unit of its sequence, that one's tiles); out: the share, then item,
# tile, off and followers of each
PROGRAM = r"""
#include <cstdio>
#include "pa_split_plan.h"
using namespace pa::split;
int main() {
  int cut, n;
  long long grid, total;
  while (scanf("%d %lld %lld %d", &cut, &grid, &total, &n) == 4) {
    const long long share = share_units(total, grid, cut != 0);
    printf("%lld", share);
    for (int k = 0; k < n; ++k) {
      long long x;
      int tiles;
      if (scanf("%lld %d", &x, &tiles) != 2) return 1;
      const Place at = place_of(x, tiles, cut != 0);
      printf(" %lld %d %d %d", at.item, at.tile, at.off, at.tile > 0 ? followers_of(tiles, at.off, share) : 0);
    }
    printf("\n");
  }
  printf("%d %d %lld\n", kItemCost, kLeastPiece, item_units(7));
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("split_plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def call(lines):
        out = subprocess.run([str(exe)], input="\n".join(lines) + "\n", check=True, capture_output=True, text=True).stdout
        return [[int(v) for v in line.split()] for line in out.strip().splitlines()]
    return call


def restated(seqs, hkv, grid, cut, units):
    """The line for the program and what it has to answer."""
    from test_split_plan import ITEM_COST, LEAST_PIECE
    share, _ = shares(seqs, hkv, grid, cut)
    total = sum(b * hkv * (t + ITEM_COST) for b, t in seqs)
    line, want = [int(cut), grid, total, len(units)], [share]
    for x in units:
        s, i, tile, off = place(x, seqs, hkv, cut)
        start = sum(b * hkv * (t + ITEM_COST) for b, t in seqs[:s])
        tiles = seqs[s][1]
        line += [x - start, tiles]
        want += [i, tile, off, 1 + (tiles - LEAST_PIECE + ITEM_COST - off) // share if tile > 0 else 0]
    return " ".join(map(str, line)), want


def test_random_batches(run):
    from test_split_plan import ITEM_COST
    rng = random.Random(7)
    lines, wants = [], []
    for _ in range(400):
        n = rng.choice([1, 1, 2, 3, 7, 20, 70])
        top = rng.choice([0, 1, 3, 8, 9, 20, 100, 600, 40000])
        seqs = [(rng.choice([1, 1, 1, 2, 5]), rng.randint(0, top)) for _ in range(n)]
        hkv, grid, cut = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 5, 16, 148, 152, 304]), rng.random() < 0.8
        share, _ = shares(seqs, hkv, grid, cut)
        total = sum(b * hkv * (t + ITEM_COST) for b, t in seqs)
        line, want = restated(seqs, hkv, grid, cut, [c * share for c in range(grid + 1) if c * share < total])
        lines.append(line)
        wants.append(want)
    assert run(lines)[:-1] == wants


def test_every_unit_of_small_items(run):
    lines, wants = [], []
    for tiles in range(0, 12):
        for cut in (True, False):
            for grid in (1, 3, 50):
                line, want = restated([(3, tiles)], 1, grid, cut, list(range(3 * (tiles + 3))))
                lines.append(line)
                wants.append(want)
    assert run(lines)[:-1] == wants


def test_the_same_constants(run):
    from test_split_plan import ITEM_COST, LEAST_PIECE
    assert run([])[-1] == [ITEM_COST, LEAST_PIECE, 7 + ITEM_COST]
