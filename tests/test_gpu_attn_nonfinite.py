"""A V scale that is not finite, in a cell that only the newest token sees: the
other rows' results are right or visibly not finite, never quietly wrong."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

BF, FP, I8 = torch.bfloat16, torch.float16, torch.int8


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("io,d", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("n", [2, 6, 8, 20, 90])
def test_a_v_scale_that_is_not_finite(n, io, d, value):
    from attn_helpers import Case, unit
    c = Case([n], [200], 4, 1, d, 16, I8, io, seed=n)
    cell = c.cells[c.table[0, 199 // 16], 199 % 16]
    cell.view(torch.float32)[2 * d // 4 + 1] = value            # K codes, V codes, K scale, V scale
    out, lse = c.forward(max_q=n)
    c.att.moe_attn_sync()
    got = out.double().cpu().numpy()
    assert not np.isfinite(got[-1]).any()
    want, want_l, mag = oa.attention(c.q64[:-1], c.k64[0][:199], c.v64[0][:199], 0, c.scale)
    assert np.abs(lse[:-1].double().cpu().numpy() - want_l).max() <= 2.0 ** -10
    ok = np.isfinite(got[:-1])
    # probabilities in fp16, an output rounded once, scores as in the other tests
    tol = (2.0 ** -9 + unit(io) * 1.01) * mag + 2.0 ** -24
    assert (np.abs(got[:-1] - want) <= tol)[ok].all()
    if n * 4 <= 32:                                             # the few-row kernel keeps the rows apart
        assert ok.all()
