"""The order of a block's copies into its ring of stages, on the host
(csrc/delta_plan.h built by the host compiler): also after a wait that gave up,
nothing is copied over a stage in use and every copy is waited for."""

import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_cached_decode_gb300", "csrc")

SOURCE = """
#include "delta_plan.h"
// events (kind, a, b): 0 a wait for stage a's parity b, 1 copies of chunk a into stage b, 2 a wait for stage a's copies of parity b
extern "C" int deliver(int n, int stages, int gives_up, int* out) {
  int k = 0, waits = 0;
  auto put = [&](int kind, int a, int b) { out[3 * k] = kind; out[3 * k + 1] = a; out[3 * k + 2] = b; ++k; };
  moe::delta_deliver(
      n, stages, [&](int st, uint32_t parity) { put(0, st, (int)parity); return ++waits != gives_up; },
      [&](int i, int st) { put(1, i, st); }, [&](int st, uint32_t parity) { put(2, st, (int)parity); });
  return k;
}
"""


@pytest.fixture(scope="module")
def deliver(tmp_path_factory):
    d = tmp_path_factory.mktemp("loader")
    src, lib = d / "loader.cpp", d / "loader.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).deliver

    def run(n, stages, gives_up=0):
        out = (ctypes.c_int * (9 * n + 30))()
        k = f(n, stages, gives_up, out)
        return [tuple(out[3 * i:3 * i + 3]) for i in range(k)]

    return run


@pytest.mark.parametrize("stages", [1, 2, 3])
@pytest.mark.parametrize("n", [0, 1, 2, 3, 4, 7, 20])
def test_copies_into_free_stages_and_waited_for(deliver, stages, n):
    for gives_up in range(0, n + 1):
        events = deliver(n, stages, gives_up)
        uses, freed, waits = [0] * stages, [0] * stages, 0
        last = {}
        for at, (kind, a, b) in enumerate(events):
            if kind == 0:
                waits += 1
                assert b == freed[a] % 2 and uses[a] == freed[a] + 1     # of the stage's use that is the last one
                if waits == gives_up:
                    assert all(e[0] == 2 for e in events[at + 1:])       # nothing is copied any more
                else:
                    freed[a] += 1
            elif kind == 1:
                assert b == a % stages and uses[b] == freed[b]           # free
                uses[b] += 1
                last[b] = a
            else:
                assert last.pop(a) // stages % 2 == b                    # its last copies, in the phase that they complete
        assert not last                                                  # and none is left under way
        if not gives_up or gives_up > max(0, n - stages):
            assert sum(e[0] == 1 for e in events) == n
