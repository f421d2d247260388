"""Sequences that go on from one window of the work space to the next, at
lengths taken from the work space's size."""

import ctypes
import os
import subprocess

import pytest
import torch

from expert_cached_decode_gb300 import GatedDelta

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_cached_decode_gb300", "csrc")


@pytest.fixture(scope="module")
def window(tmp_path_factory):
    """Chunks of a window, by the library's own arithmetic."""
    d = tmp_path_factory.mktemp("window")
    src, lib = d / "window.cpp", d / "window.so"
    src.write_text('#include "delta_plan.h"\nextern "C" int window(int hk, int hv, int dk) { return moe::delta_window(hk, hv, dk); }\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib)).window


def _rule64(q, k, v, g, beta, state, scale):
    """One head in 64 bits on the GPU: q, k [n, dk], v [n, dv], g, beta [n] -> outputs, state."""
    q, k = (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    out, S = torch.empty_like(v), state.clone()
    e = g.exp()
    for t in range(len(v)):
        S *= e[t]
        u = beta[t] * (v[t] - k[t] @ S)
        S += torch.outer(k[t], u)
        out[t] = scale * (q[t] @ S)
    return out, S


@pytest.mark.parametrize("hk,hv,dk,dv,dtype", [(64, 128, 128, 128, HF), (64, 128, 64, 64, BF), (32, 64, 128, 64, BF)])
def test_a_state_that_goes_on_in_the_next_window(window, hk, hv, dk, dv, dtype):
    W = window(hk, hv, dk)
    # each ends in the first chunk behind a border
    lens = [64 * W + 30, 64 * W]
    bases, t0 = [], 0
    for s, n in enumerate(lens):
        bases.append(t0 // 64 + s)
        t0 += n
    ends = [b + -(-n // 64) - 1 for b, n in zip(bases, lens)]
    assert ends[0] == W and bases[1] // W == 1 and ends[1] // W == 2       # both cross a border
    n = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(hv + dk)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    q, k, v = rand(n, hk, dk).to(dtype), rand(n, hk, dk).to(dtype), rand(n, hv, dv).to(dtype)
    decay, beta = -torch.rand(n, hv, device="cuda", generator=g) * 0.002, torch.rand(n, hv, device="cuda", generator=g) * 0.2
    first = rand(2, hv, dk, dv)
    state, out = first.clone(), torch.empty(n, hv, dv, dtype=dtype, device="cuda")
    cu = torch.tensor([0, lens[0], n], dtype=torch.int32, device="cuda")
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    op = GatedDelta(hk, hv, dk, dv, dtype=dtype)
    op.moe_delta_forward(q, k, v, decay, beta, state, out, cu, slots, slots)
    op.moe_delta_sync()
    for s, h in ((0, 0), (0, hv - 1), (1, hv // 2)):
        a, b = int(cu[s]), int(cu[s + 1])
        r, hq = slice(a, b), h // (hv // hk)
        o, S = _rule64(*(x[r, i].double() for x, i in ((q, hq), (k, hq), (v, h), (decay, h), (beta, h))), first[1 - s, h].double(), dk ** -0.5)
        # 2^-17 of the state's length: far above what 22 bits make of it, far below what a border that loses it does (most of it)
        assert (state[1 - s, h].double() - S).norm() <= 2.0 ** -17 * S.norm()
        # rounding (2^-8 or 2^-11 of a value) and products of 11 bits, as one length: a row of outputs adds up errors by chance
        assert ((out[r, h].double() - o).norm(dim=1) <= 2.0 ** -7 * o.norm(dim=1) + 2.0 ** -20).all()
