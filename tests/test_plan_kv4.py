"""The 4-bit attention's choice of a range length (csrc/kv4_plan.h), compiled
for the host and checked against the least length found one by one (CPU
only)."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GRID = 152  # CTAs of head dims 128 and 256 on 152 SMs

SRC = r"""
#include "kv4_plan.h"
using namespace hy::kv4;
// bounds, and the first of 32 candidates whose ranges fit, as a warp finds it (0: none)
extern "C" unsigned choose(const unsigned* n, unsigned nb, unsigned nkv, unsigned grid, unsigned W, unsigned* lo,
                           unsigned* hi) {
  unsigned total = 0, items = 0;
  for (unsigned b = 0; b < nb; ++b) {
    total += nkv * n[b];
    items += n[b] ? nkv : 0;
  }
  *lo = shortest_range(total, grid, W);
  *hi = longest_range(total, grid, items, *lo);
  for (unsigned lane = 0; lane < 32; ++lane) {
    const unsigned m = range_length(*lo, *hi, lane);
    unsigned ranges = 0;
    for (unsigned b = 0; b < nb; ++b) ranges += ranges_of(n[b], m, 1.0f / (float)m);
    if (nkv * ranges <= grid) return m;
  }
  return 0;
}
extern "C" unsigned candidate(unsigned lo, unsigned hi, unsigned i) { return range_length(lo, hi, i); }
extern "C" unsigned ranges(unsigned x, unsigned m) { return ranges_of(x, m, 1.0f / (float)m); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "bandwidth_bound_hybrid_gb300", "csrc"),
                    str(d / "plan.cpp"), "-o", str(d / "plan.so")], check=True)
    return ctypes.CDLL(str(d / "plan.so"))


def choose(plan, n, nkv, grid, W):
    lo, hi = ctypes.c_uint(0), ctypes.c_uint(0)
    m = plan.choose((ctypes.c_uint * len(n))(*n), len(n), nkv, grid, W, ctypes.byref(lo), ctypes.byref(hi))
    return m, lo.value, hi.value


def least(n, nkv, grid, lo, hi):
    return next(m for m in range(lo, hi + 1) if nkv * sum(-(-x // m) for x in n) <= grid)


def draws(seed, count, top):
    rng = random.Random(seed)
    while count:
        nkv = rng.choice([1, 2, 4, 8])
        n = [rng.randint(1, top) if rng.random() < 0.95 else 0 for _ in range(rng.randint(1, 8))]
        W, grid = rng.choice([8, 12]), rng.choice([GRID, 2 * GRID])
        if 0 < nkv * sum(x > 0 for x in n) <= grid and nkv * sum(-(-x // W) for x in n) > grid:
            count -= 1
            yield n, nkv, grid, W


def test_ragged_batches_of_medium_contexts_take_the_least_length(plan):
    """8 sequences of 1k-16k rows over 2 kv heads x 256 (tiles of 16 rows, 8 warps)."""
    rng = random.Random(0)
    for _ in range(200):
        n = [rng.randint(1024, 16384) // 16 + 1 for _ in range(8)]
        m, lo, hi = choose(plan, n, 2, GRID, 8)
        assert hi - lo <= 31 and m == least(n, 2, GRID, lo, hi), (n, m, lo, hi)


def test_least_of_the_candidates(plan):
    for n, nkv, grid, W in draws(1, 2000, 4000):
        m, lo, hi = choose(plan, n, nkv, grid, W)
        best = least(n, nkv, grid, lo, hi)
        assert best <= m <= best + max(-(-(hi - lo) // 31) - 1, 0), (n, nkv, grid, W, m, best)  # exact for close bounds


def test_candidates_span_the_bounds(plan):
    plan.candidate.restype = ctypes.c_uint
    for d in [*range(0, 100), 1000, 2 ** 30 - 1, 2 ** 31]:
        c = [plan.candidate(5, 5 + d, i) for i in range(32)]
        assert c[0] == 5 and c[31] == 5 + d and c == sorted(c)
        assert max(b - a for a, b in zip(c, c[1:])) <= -(-d // 31)
        if d <= 31:
            assert set(c) == set(range(5, 6 + d))


def test_ranges_are_rounded_up(plan):
    rng = random.Random(2)
    plan.ranges.restype = ctypes.c_uint
    for _ in range(20000):
        m = rng.randint(1, 10 ** rng.randint(1, 6))
        x = min(m * rng.randint(0, 3000) + rng.randint(-1, 1), 2 ** 30)
        if x >= 0:
            assert plan.ranges(x, m) == -(-x // m), (x, m)
