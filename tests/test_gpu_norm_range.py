"""The norms where a value times its gate is beyond fp32 and the normed value's
is not."""

import numpy as np
import pytest
import torch

from delta_helpers import unit
from expert_cached_decode_gb300 import moe_norm_block, moe_norm_gated
from oracle import delta as od

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _f(t):
    return t.double().cpu().numpy()


def test_products_that_pass_fp32_on_the_way():
    # |o act(z)| and |y gate| are beyond fp32, the normed values times them are not
    d = 128
    g = np.random.default_rng(0)
    o = torch.from_numpy(np.sign(g.standard_normal((3, 1, d))) * (1 + g.random((3, 1, d)))).to(BF).cuda() * 2.0 ** 59
    z = torch.full((3, 1, d), 2.0 ** 70, dtype=BF, device="cuda")
    w, out = torch.full((d,), 0.5, dtype=BF, device="cuda"), torch.empty_like(o)
    moe_norm_gated(o, z, w, out)
    want = od.norm_gated(_f(o), _f(z), _f(w), "silu", False, 1e-6, 0.0)
    assert (np.abs(_f(out) - want) <= (unit(BF) + 2.0 ** -19) * np.abs(want)).all()
    y, gate, h, x = o.view(3, d), z.view(3, d), torch.empty(3, d, device="cuda"), torch.empty(3, d, dtype=BF, device="cuda")
    for act in ("none", "silu"):
        moe_norm_block(y, None, h, x, pre_w=w, post_w=w, gate=gate, act=act, scale=2.0 ** -20)
        want, wx = od.norm_block(_f(y), None, _f(gate), _f(w), _f(w), act, 2.0 ** -20, 1e-6, 0.0)
        assert (np.abs(_f(h) - want) <= 2.0 ** -19 * np.abs(want)).all()
        assert (np.abs(_f(x) - wx) <= (unit(BF) + 2.0 ** -19) * np.abs(wx)).all()
