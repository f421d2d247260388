"""The gated delta rule with decays above 1 (g > 0: the state grows), in chunks
and token by token, against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from delta_helpers import Case

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

# The bounds are those of Case.check: its magnitudes grow with the state, and in chunks Z and U are kept under a power of two
# per token that takes the growth out, so that they hold the bits that they hold without it.


def _case(lens, dtype, g, aligned, dk=128, dv=128, **kw):
    c = Case(lens, dk=dk, dv=dv, dtype=dtype, seed=len(lens) + dk, pad=2, **kw)
    c.g64[:] = np.broadcast_to(np.float32(g), c.g64.shape).astype(np.float64)
    if aligned:                                # keys that are the queries: q.k at its largest
        c.x[:, :c.nq] = c.x[:, c.nq:2 * c.nq]
        c.x64 = c.x.double().cpu().numpy()
    return c


@pytest.mark.parametrize("n", [25, 64, 200])
@pytest.mark.parametrize("dtype,g", [(BF, 0.05), (BF, 0.2), (HF, 0.02), (HF, 0.05)])
@pytest.mark.parametrize("aligned", [False, True])
def test_the_state_grows(n, dtype, g, aligned):
    # (fp16 outputs: growth that keeps them below 65,504)
    c = _case([n, n + 3], dtype, g, aligned, fresh=(0,))
    d = c.forward()
    c.check(d)
    c.op.moe_delta_sync()
    c.check(c.forward(max_q=1))                # the same token by token


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128)])
def test_the_state_grows_in_every_layout(dk, dv):
    c = _case([130, 1, 40], BF, 0.1, True, dk=dk, dv=dv)
    c.check(c.forward())


@pytest.mark.parametrize("aligned", [False, True])
def test_growth_and_decay_in_one_chunk(aligned):
    # up by 2^14 and down again, one large step, a token that forgets all and growth behind it; heads apart from each other
    n = 150
    g = np.zeros((n + 2, 4))
    g[:, 0] = np.where(np.arange(n + 2) % 40 < 20, 0.5, -0.5)
    g[17, 1] = 9.0
    g[18:, 1] = -0.15
    g[:, 2] = 0.1
    g[30, 2] = -np.inf
    g[100, 2] = -np.inf
    g[:, 3] = -0.05                            # (nothing grows)
    c = _case([n], BF, g, aligned)
    c.check(c.forward())
    c.check(c.forward(max_q=1))


def test_a_head_that_does_not_grow_keeps_its_bits():
    # growth of one head changes no other one's results
    c = Case([200, 70], seed=3)
    want = c.forward()
    c.g64[:, 1] = np.float32(0.1)
    got = c.forward()
    torch.cuda.synchronize()
    for name, h in (("out", 1), ("state", 1)):
        a, b = want[name].clone(), got[name].clone()
        a[:, h] = 0
        b[:, h] = 0
        assert torch.equal(a, b)
    c.check(got)
