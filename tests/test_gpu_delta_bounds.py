"""The two bounds of the next state in chunks: from the tokens' steps where none of
them lengthens a column, else from sums over T; and chunks of both kinds in turn."""

import numpy as np
import pytest
import torch

from delta_helpers import Case
from oracle import delta as od

pytestmark = pytest.mark.gpu


def _check(c, n):
    # 2^-17 of the state's length, as for states of chunks elsewhere: 22 bits and some ten operands make 2^-19 of it, and a step
    # with |1 - beta |k^|^2| up to 2 along one of 128 random directions lengthens an error by less than it does the state
    q, k, v = c.views(c.x64)
    o, S, mag, size = od.rule(q[:n], k[:n], v[:n], c.g64[:n], c.b64[:n], c.st64[c.s_in[0]], c.scale, c.normalize)
    for max_q in (None, 1):
        d = c.forward(max_q=max_q)
        torch.cuda.synchronize()
        st, out = d["state"][int(c.s_out[0])].double().cpu().numpy(), d["out"].double().cpu().numpy()[:n]
        assert np.linalg.norm(st - S) <= 2.0 ** -17 * np.linalg.norm(S)
        assert np.linalg.norm(out - o) <= 2.0 ** -8 * np.linalg.norm(o)        # (a rounding to bf16 is 2^-9.3 of a length by chance)
    c.op.moe_delta_sync()


@pytest.mark.parametrize("n", [64, 130, 1700])
@pytest.mark.parametrize("lo,hi", [(-1.0, 3.0), (0.0, 2.0), (2.0, 2.0), (-0.2, 0.0)])
def test_beta_of_every_size(n, lo, hi):
    c = Case([n], hk=1, hv=2, seed=n, keep=(0,), decay=0.05)
    c.b64 = (lo + (hi - lo) * np.random.default_rng(n).random(c.b64.shape)).astype(np.float32).astype(np.float64)
    _check(c, n)


@pytest.mark.parametrize("n", [130, 1700])
def test_keys_longer_than_one(n):
    c = Case([n], hk=1, hv=2, seed=n, normalize=False, keep=(0,), decay=0.05)
    c.x[:, c.nq:2 * c.nq] *= 1.4                       # beta |k|^2 up to 2
    c.x64 = c.x.double().cpu().numpy()
    _check(c, n)


def test_chunks_of_both_kinds_in_turn():
    n = 500
    c = Case([n], hk=1, hv=2, seed=4, keep=(0,), decay=0.05)
    c.b64[70] = 2.5                                    # in the second chunk, for both heads
    c.b64[200:210, 1] = -0.5
    c.b64[450, 0] = 2.5
    _check(c, n)
