"""Gates far below zero, where the logistic function and silu are small numbers
of their own."""

import numpy as np
import pytest
import torch

from delta_helpers import unit
from expert_cached_decode_gb300 import GatedDelta, moe_norm_block, moe_norm_gated
from oracle import delta as od

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
Z = [-0.5, -5.0, -20.0, -60.0, -87.0, -88.0, 3.0, 20.0, 88.0, 0.0]


def _f(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("full", [False, True])
def test_block_gates_in_fp32(act, full):
    # An exponential of 2 units in the last place, a sum, a quotient and two products are below 2^-21.  No absolute slack but the
    # steps of fp32's smallest numbers: below 2^-126 numbers are multiples of 2^-149, so that rounding is off by 2^-150 there, once
    # in the gate (then times 88 and y at most) and once in the result (y 1.6e-38 at -87 is such a number wherever |y| < 0.7).
    n, d = len(Z), 64
    y = torch.randn(n, d, device="cuda")
    gate = torch.tensor(Z, device="cuda").to(BF)[:, None]
    gate = gate.expand(n, d).contiguous() if full else gate
    h = torch.empty(n, d, device="cuda")
    moe_norm_block(y, None, h, gate=gate, act=act)
    want = _f(y) * od.act(_f(gate), act)
    assert (np.abs(_f(h) - want) <= 2.0 ** -21 * np.abs(want) + (np.abs(_f(y)) * 88 + 1) * 2.0 ** -149).all()


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_norm_gates(act):
    # bf16 has fp32's range: one rounding, and 2^-16 of the result for an exponential whose error grows with -z (95 units at -80)
    n, d = len(Z), 128
    o = torch.randn(n, 1, d, device="cuda").to(BF)
    z = torch.tensor(Z, device="cuda").to(BF)[:, None, None].expand(n, 1, d).contiguous()
    w, out = torch.ones(d, dtype=BF, device="cuda"), torch.empty_like(o)
    moe_norm_gated(o, z, w, out, act=act)
    want = od.norm_gated(_f(o), _f(z), _f(w), act, False, 1e-6, 0.0)
    assert (np.abs(_f(out) - want) <= (unit(BF) + 2.0 ** -16) * np.abs(want) + 2.0 ** -133).all()


def test_convolution_gates():
    # y = silu(x): the newest tap alone
    op = GatedDelta(1, 1, 64, 64, taps=2)
    n, C = len(Z), op.channels
    x = torch.tensor(Z, device="cuda").to(BF)[:, None].expand(n, C).contiguous()
    w = torch.tensor([0.0, 1.0], device="cuda").to(BF).expand(C, 2).contiguous()
    y, state = torch.empty_like(x), torch.zeros(1, 1, C, dtype=BF, device="cuda")
    cu, slot = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    op.moe_delta_prepare(x, w, None, state, y, None, None, None, None, None, None, cu, slot, slot)
    want = od.act(_f(x), "silu")
    assert (np.abs(_f(y) - want) <= (unit(BF) + 2.0 ** -16) * np.abs(want) + 2.0 ** -133).all()


@pytest.mark.parametrize("h", [F, BF])
@pytest.mark.parametrize("act,want", [("sigmoid", [1.0, 0.0, 1.0, 0.0, 1.0, 0.0]), ("silu", [np.inf, np.nan, 1e30, 0.0, 300.0, 0.0])])
def test_gates_without_end(h, act, want):
    z = torch.tensor([np.inf, -np.inf, 1e30, -1e30, 300.0, -300.0, np.nan], device="cuda").to(BF)[:, None]
    y = torch.ones(7, 64, device="cuda")
    out = torch.empty(7, 64, dtype=h, device="cuda")
    moe_norm_block(y, None, out, gate=z, act=act)
    want = torch.tensor(want + [np.nan], dtype=torch.float64)
    got = out[:, 5].double().cpu()
    assert torch.allclose(got, want.to(BF).double(), rtol=2.0 ** -7, atol=0, equal_nan=True), got
    w, o, g = torch.ones(64, dtype=BF, device="cuda"), torch.ones(7, 1, 64, dtype=BF, device="cuda"), z[:, None].expand(7, 1, 64).contiguous()
    res = torch.empty_like(o)
    moe_norm_gated(o, g, w, res, act=act, eps=0.0)
    assert torch.allclose(res[:, 0, 5].double().cpu(), want.to(BF).double(), rtol=2.0 ** -7, atol=0, equal_nan=True), res[:, 0, 5]
