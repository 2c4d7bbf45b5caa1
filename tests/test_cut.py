"""How the SMs are shared out between the two parts of the shared-prefix call, on the CPU.

hs_cut.h is host code: a small program prints the pairs of SMs that the own rows' part gets."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hierarchical_kv_cache_hs_gb300", "csrc")
ALL = 76

MAIN = r"""
#include <cstdio>
#include "hs_cut.h"
int main() {
    int e4m3, batch, positions, heads, listed, rows, prefix, ragged, all;
    static int32_t entry;
    while (std::scanf("%d %d %d %d %d %d %d %d %d", &e4m3, &batch, &positions, &heads, &listed, &rows, &prefix, &ragged, &all) == 9) {
        hs_attend_t a = {};
        a.row_format = e4m3 ? HS_ROWS_E4M3 : HS_ROWS_16BIT;
        a.batch = batch, a.positions = positions, a.heads = heads;
        a.n_rows = a.entries = rows;
        (listed ? a.slots : a.lengths) = &entry;
        const int units = (int)(((int64_t)batch * positions * heads + 127) / 128);
        std::printf("%d\n", hs_attn::pairs_beside(a, ragged, units, (int)hs_attn::Cut::tiles_of(prefix, 128), all));
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def pairs(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("cut")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    str(at / "main.cpp"), "-o", str(at / "main")], check=True)

    def ask(cases):
        text = "".join(" ".join(str(int(x)) for x in c) + "\n" for c in cases)
        r = subprocess.run([str(at / "main")], input=text, capture_output=True, text=True, timeout=120, check=True)
        return [int(x) for x in r.stdout.split()]
    return ask


def _up(a, b):
    return -(-a // b)


def _in_pieces(e4m3, batch, positions, heads, rows, n):
    """Whether n pairs would cut the own rows' units: whole ones, or a line of equal pieces where those are shorter
    by more than their join's time."""
    narrow = e4m3 and heads <= 32
    units, tiles = batch * positions * _up(heads, 128), max(1, _up(rows, 64))
    workers = min(2 * n if narrow else n, units * tiles)
    return _up(units, workers) * tiles > _up(units * tiles, workers) + (6 if narrow else 10)


def test_some_pairs_take_whole_units_only(pairs):
    """Else the join of the pieces would stand between the own rows' kernel and the prefix's."""
    rng = random.Random(5)
    cases = []
    while len(cases) < 4000:
        batch, positions = int(2 ** rng.uniform(0, 8.5)), rng.choice((1, 1, 1, 2, 3, 7))
        heads, rows = rng.choice((1, 8, 16, 20, 32, 33, 64, 128, 200)), int(2 ** rng.uniform(0, 14))
        c = (rng.random() < 0.5, batch, positions, heads, rng.random() < 0.7, rows, int(2 ** rng.uniform(0, 17)), rng.random() < 0.3,
             rng.choice((ALL, ALL, 66, 2, 1)))
        if batch * positions * heads <= 152 * 128:
            cases.append(c)
    beside = 0
    for c, n in zip(cases, pairs(cases)):
        e4m3, batch, positions, heads, listed, rows, _, _, all_pairs = c
        assert 1 <= n <= all_pairs
        if n < all_pairs:
            beside += 1
            assert not _in_pieces(e4m3, batch, positions, heads, rows, n), (c, n)
            assert listed or rows <= 512
    assert beside > 500


@pytest.mark.parametrize("case", [
    # 8 bits, requests, positions, heads, lists, entries, prefix: 49 to 80 us beside the prefix, 43 to 60 with all pairs first
    (1, 1, 1, 16, 1, 2048, 3001), (1, 1, 1, 16, 1, 2048, 16384), (1, 4, 1, 16, 1, 2048, 3001), (1, 8, 1, 16, 1, 2048, 4096),
    (1, 16, 1, 16, 1, 2048, 3001), (1, 5, 3, 20, 1, 2048, 3001), (0, 1, 1, 16, 1, 2048, 3001), (0, 1, 1, 128, 1, 2048, 3001),
    (1, 1, 1, 128, 1, 2048, 3001), (1, 1, 1, 16, 1, 1024, 3001)])
def test_few_requests_with_long_lists_take_all_pairs_first(pairs, case):
    assert pairs([case + (0, ALL)]) == [ALL]


@pytest.mark.parametrize("case,low,high,first", [
    # the same, the pairs within a few percent of the best of a sweep, and all of them first: us at best, and so
    ((0, 8, 1, 128, 1, 2048, 16384), 8, 12, (55, 71)),
    ((0, 8, 1, 16, 1, 1024, 3001), 8, 20, (36, 49)),
    ((0, 64, 1, 16, 1, 2048, 16384), 32, 32, (92, 94)),
    ((1, 64, 1, 16, 1, 2048, 16384), 32, 32, (75, 100)),
    ((1, 64, 1, 16, 1, 1024, 16384), 32, 36, (73, 88)),
    ((1, 8, 1, 16, 0, 500, 65536), 4, 16, (65, 82)),
    ((0, 64, 1, 16, 0, 512, 16384), 22, 30, (53, 57))])
def test_units_that_fit_run_beside_the_prefix(pairs, case, low, high, first):
    n = pairs([case + (0, ALL)])[0]
    assert low <= n <= high or (n == ALL and first[1] <= 1.05 * first[0])
