"""The attention kernels' index arithmetic on the host (csrc/attn_plan.h built
by the host compiler): which rows of a call see a run of cells, at lengths,
windows and group sizes up to the ones that the entry points accept, the size
of an eviction's copy, and the registers that a block's roles take together."""

import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_cached_decode_gb300", "csrc")

SOURCE = """
#include "attn_plan.h"
extern "C" void rows_that_see(int j0, int cells, int n, int len, int window, int g, int* ab) {
  const moe::RowSpan r = moe::rows_that_see(j0, cells, n, len, window, g);
  ab[0] = r.a;
  ab[1] = r.b;
}
extern "C" int evict_copy_blocks(int budget, int max_len, int cells) {
  return moe::evict_copy_blocks(budget, max_len, cells);
}
extern "C" void roles(int* out) {
  out[0] = moe::ChunkRoles::Block::kThreads;
  out[1] = moe::ChunkRoles::Block::registers();
  out[2] = moe::WeightRoles::Block::kThreads;
  out[3] = moe::WeightRoles::Block::registers();
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def _span(plan, *args):
    ab = (ctypes.c_int * 2)()
    plan.rows_that_see(*args, ab)
    return ab[0], ab[1]


def _want(j0, cells, n, length, window, g):
    """From the mask: token i, in cell p = length - n + i, sees the cells p - window < j <= p (without limits on size)."""
    base = length - n
    lo = max(0, j0 - base)                                       # p >= the first cell
    hi = min(n, j0 + cells - 1 + window - base) if window else n   # p - window < the last cell
    return (lo * g, hi * g) if lo < hi else None


def _check(plan, *args):
    a, b = _span(plan, *args)
    want = _want(*args)
    assert 0 <= a <= b <= args[2] * args[5], (args, a, b)
    if want is None:
        assert a == b, (args, a, b)
    else:
        assert (a, b) == want, (args, a, b)


@pytest.mark.parametrize("cells", [64, 256])
@pytest.mark.parametrize("g", [1, 3, 8, 32])
@pytest.mark.parametrize("window", [1, 5, 4096])
@pytest.mark.parametrize("length", [2 ** 26, 2 ** 26 + 64 * 33, 2 ** 27, 2 ** 28 + 999, 2 ** 30 - 1])
def test_cells_far_before_the_window(plan, cells, g, window, length):
    # first - window times the group passes 32 bits
    for n in (1, 2, 40, 5000):
        for j0 in (0, cells, 3 * cells, length // 2 // cells * cells, (length - 1) // cells * cells,
                   max(0, (length - n - window) // cells * cells)):
            _check(plan, j0, cells, n, length, window, g)


def test_spans_against_the_mask_itself(plan):
    rng = random.Random(0)
    for _ in range(3000):
        n, length, g = rng.randint(0, 40), rng.randint(1, 300), rng.choice([1, 2, 5])
        window, cells = rng.choice([0, 0, 1, 7, 100]), rng.choice([64, 16])
        j0 = rng.randrange(length) // cells * cells
        seen = [i for i in range(n) if any(j <= length - n + i and (not window or j > length - n + i - window)
                                           for j in range(j0, j0 + cells))]
        a, b = _span(plan, j0, cells, n, length, window, g)
        assert [i for i in range(n) if a <= i * g < b] == seen
        if window == 0:
            _check(plan, j0, cells, n, length, window, g)


def test_spans_over_the_whole_range(plan):
    rng = random.Random(1)
    for _ in range(20000):
        length = rng.randint(1, 2 ** rng.randint(1, 30) - 1)
        n, cells = rng.randint(0, min(2 ** 24, 2 ** rng.randint(0, 24))), rng.choice([64, 256])
        window = rng.choice([0, 1, rng.randint(1, max(1, length - 1))])
        _check(plan, rng.randrange(length) // cells * cells, cells, n, length, window, rng.choice([1, 7, 8, 32]))


def test_registers_of_every_warpgroup_are_counted(plan):
    # warpgroups x 128 threads x their shares: 2 softmax, cells, products; 4 that add up, loads, products
    out = (ctypes.c_int * 4)()
    plan.roles(out)
    assert list(out) == [512, 128 * (2 * 152 + 96 + 96), 768, 128 * (4 * 88 + 64 + 64)]
    # what the launch bounds leave a thread (65,536 registers a block, in steps of 8) covers them
    for threads, registers in ((out[0], out[1]), (out[2], out[3])):
        assert 65536 // threads // 8 * 8 * threads >= registers


@pytest.mark.parametrize("budget", [1, 63, 64, 65, 2 ** 20 + 1, 2 ** 30, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 1])
@pytest.mark.parametrize("max_len", [0, 1, 64, 100, 2 ** 20, 2 ** 30 - 1])
def test_blocks_of_an_evictions_copy(plan, budget, max_len):
    # every cell that can be kept, and no block beyond them (one where nothing can: a launch has to have blocks)
    assert plan.evict_copy_blocks(budget, max_len, 64) == max(1, -(-min(budget, max_len) // 64))
