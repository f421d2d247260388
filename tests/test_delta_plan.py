"""Index arithmetic of the gated delta rule's chunks on the host
(csrc/delta_plan.h built by the host compiler): chunk numbers, parts, and the
registers that a block's roles take."""

import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_cached_decode_gb300", "csrc")

SOURCE = """
#include "delta_plan.h"
extern "C" int base(int t0, int s) { return moe::delta_chunk_base(t0, s); }
extern "C" void parts(int n, int most, int front, int* out) {
  const moe::DeltaParts p = moe::delta_parts(n, most, front);
  out[0] = p.parts;
  out[1] = p.first;
  out[2] = p.len;
}
extern "C" int pass1(int parts, int dk, int dv) { return moe::delta_pass1_blocks(parts, dk, dv); }
extern "C" void cut(int n_seqs, int hv, int dk, int dv, int longest, int sms, int cuts, int most, int* out) {
  const moe::DeltaCut c = moe::delta_cut(n_seqs, hv, dk, dv, longest, sms, cuts, most);
  out[0] = c.parts;
  out[1] = c.front;
}
extern "C" int ordered(int n_seqs, int hv, int sms) { return moe::delta_ordered(n_seqs, hv, sms); }
extern "C" void roles(int* out) {
  out[0] = moe::DeltaRoles::Block::kThreads;
  out[1] = moe::DeltaRoles::Block::registers();
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def test_chunks_have_numbers_of_their_own(plan):
    g = random.Random(0)
    for _ in range(300):
        lens = [g.choice([0, 1, 63, 64, 65, g.randrange(1000)]) for _ in range(g.randrange(1, 40))]
        t0, last = g.choice([0, 0, 5, 64, 100]), -1
        total = t0 + sum(lens) + g.choice([0, 7])
        for s, n in enumerate(lens):
            b = plan.base(t0, s)
            if n:
                assert b > last                              # ascending, and none twice
                last = b + -(-n // 64) - 1
                assert last < total // 64 + len(lens)        # the number that the windows go through
            t0 += n


def test_parts_cover_a_sequence(plan):
    out = (ctypes.c_int * 3)()
    for most in (1, 3, 4, 7, 16):
        for front in (1, 2, 3, 9, 100, 500):
            for n in list(range(1, 400)) + [1000, 4097]:
                plan.parts(n, most, front, out)
                parts, first, length = out
                assert 1 <= parts <= most and parts != 2     # pass 1 finds the first part and all between, so two make no sense
                assert parts > 1 or first == n
                assert parts == 1 or n >= 24
                assert first + (parts - 2) * length < n <= first + (parts - 1) * length   # the last part is not empty


def test_cut_calls_fit_the_buffers_and_the_machine(plan):
    out = (ctypes.c_int * 2)()
    for seqs in (1, 2, 5, 40, 4096):
        for hv in (1, 3, 8, 32, 128):
            for dk in (64, 128):
                for dv in (64, 128):
                    for longest in (1, 23, 24, 60, 192, 1 << 18):
                        plan.cut(seqs, hv, dk, dv, longest, 152, 320, 16, out)
                        p, front = out
                        assert 1 <= p <= 16 and p != 2 and front >= 1
                        if longest < 24:
                            assert p == 1
                        if p > 1:
                            # the host allocates 320 // hv (sequence, part) pairs
                            assert seqs * p <= 320 // hv
                            # the first parts' blocks and those that find M and N beside them, in `front` waves
                            chains = seqs * hv
                            assert chains < 152 and chains * (plan.pass1(p, dk, dv) - 1) <= front * (152 - chains)


def test_the_roles_registers_fit_a_block(plan):
    out = (ctypes.c_int * 2)()
    plan.roles(out)
    assert out[0] == 512 and out[1] <= 65536


def test_blocks_are_ordered_where_there_is_a_choice(plan):
    assert plan.ordered(9, 32, 152) and plan.ordered(128, 2, 152)
    # one sequence, an SM for every block, and more sequences than a block's threads rank
    assert not plan.ordered(1, 128, 100) and not plan.ordered(19, 8, 152) and not plan.ordered(129, 128, 152)
