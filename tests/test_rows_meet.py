"""Whether strided rows reach into a run of bytes (csrc/rows.h built by the host
compiler), against every byte looked at."""

import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_cached_decode_gb300", "csrc")

SOURCE = """
#include "rows.h"
extern "C" int meet(int64_t a, int64_t rows, int64_t stride, int64_t width, int64_t b, int64_t n) {
  return moe::rows_meet(moe::Rows{(const void*)a, rows, stride, width}, moe::bytes_at((const void*)b, n));
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src, lib = d / "rows.cpp", d / "rows.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).meet
    f.argtypes = [ctypes.c_int64] * 6
    return lambda *a: bool(f(*a))


def test_every_byte(meet):
    g = random.Random(0)
    seen = set()
    for _ in range(20000):
        rows, width = g.randrange(0, 6), g.randrange(0, 9)
        stride = width + g.choice([0, 0, 1, 5, 30])
        a, b, n = 1000 + g.randrange(80), 1000 + g.randrange(160), g.randrange(0, 40)
        mine = {a + r * stride + i for r in range(rows) for i in range(width)}
        want = bool(mine & set(range(b, b + n)))
        assert meet(a, rows, stride, width, b, n) == want, (a, rows, stride, width, b, n)
        seen.add((want, rows > 1 and a < b and b + n < a + (rows - 1) * stride))
    assert len(seen) == 4                              # both answers, between the rows and not


def test_far_apart_and_none(meet):
    far = 2 ** 40
    assert not meet(4096, 2 ** 24, far, 64, 4096 + 64, far - 64)            # all that lies between the first two rows
    assert meet(4096, 2 ** 22, far, 64, 4096 + 64, far - 63)
    assert meet(4096, 2 ** 22, far, 64, 4096 + (2 ** 22 - 1) * far + 63, 1) and not meet(4096, 2 ** 22, far, 64, 4096 + (2 ** 22 - 1) * far + 64, 1)
    assert not meet(0, 4, 16, 16, 0, 64) and not meet(4096, 4, 16, 16, 0, 1 << 40)      # NULL
    assert meet(4096, 1000, 0, 2, 4097, 8) and not meet(4096, 1000, 0, 2, 4098, 8)      # the same bytes again and again
