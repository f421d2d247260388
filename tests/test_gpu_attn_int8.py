"""Attention over int8 cells at the precision that its products have:
probabilities in fp16 below a reference that follows the scores and the V
scales, in every kernel, where few cells are seen (a rounding is not averaged
out), where the reference grows within a tile, and with V scales that differ
from cell to cell."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

BF, FP, I8 = torch.bfloat16, torch.float16, torch.int8


def _case(n, lens, hq, hkv, d, page, io, **kw):
    from attn_helpers import Case
    return Case(n, lens, hq, hkv, d, page, I8, io, **kw)


def _scale_values(c, factor):
    """V of cell j of sequence s times factor(s, j) [hkv], a power of two, in the cells and in the 64-bit values."""
    off = 2 * c.hkv * c.d + 4 * c.hkv
    for s, length in enumerate(c.kv_lens):
        j = np.arange(length)
        f = np.stack([factor(s, i) for i in j]).astype(np.float32).reshape(length, c.hkv)
        page = torch.from_numpy(c.table[s, j // c.page].astype(np.int64)).cuda()
        slot = torch.from_numpy(j % c.page).cuda()
        vs = c.cells[page, slot, off:off + 4 * c.hkv].contiguous().view(torch.float32)
        c.cells[page, slot, off:off + 4 * c.hkv] = (vs * torch.from_numpy(f).cuda()).view(torch.uint8)
        c.v64[s] = c.v64[s] * f[..., None]


def _check(c, **kw):
    """As attn_helpers.check_forward, with probabilities in fp16: each is rounded to 2^-11 of itself or, below fp16's
    normal numbers, to 2^-25 in units of the reference.  That lies 2^7 (many rows; 2^15 with few) below the largest score
    plus the largest scale's exponent, both rounded up, so a step of it is at most 2^-30 of the largest |v|; twice,
    because a reference that grows inside a tile rounds once more."""
    from attn_helpers import score_error, unit
    out, lse = c.forward(**kw)
    c.att.moe_attn_sync()
    got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for s in range(len(c.kv_lens)):
        r = c.rows(s)
        want, want_l, mag = oa.attention(c.q64[r], c.k64[s], c.v64[s], c.window, c.scale)
        es = score_error(c, s)
        assert np.abs(got_l[r] - want_l).max(initial=0.0) <= 2 * es + 2.0 ** -21 * np.abs(want_l).max(initial=0.0) + 2.0 ** -20
        tiny = 2.0 ** -29 * c.kv_lens[s] * np.abs(c.v64[s]).max(initial=0.0)
        tol = (2.0 ** -11 * 1.01 + 2 * es + 2.0 ** -18) * mag + tiny + unit(c.dtype) * 1.01 * np.abs(want) + 2.0 ** -24
        bad = np.abs(got[r] - want) > tol
        assert not bad.any(), (s, np.argwhere(bad)[:5], (np.abs(got[r] - want) / tol).max())


# rows per K/V head: 8 and 32 (few rows), 80 (two streams on alternate tiles), 400 (two halves of a row tile)
ROWS = [1, 4, 10, 50]


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 5])
@pytest.mark.parametrize("n", ROWS)
def test_rows_that_see_few_cells(io, d, window, n):
    _check(_case([n, n], [n + 3, 300], 8, 1, d, 16, io, window=window, seed=n + window), max_q=n)


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("n", ROWS)
def test_references_that_grow(io, n):
    _check(_case([n, n], [700, 130], 8, 1, 128, 32, io, seed=n, std=4.0), max_q=n)


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", ROWS)
def test_scales_that_differ_from_cell_to_cell(io, d, n):
    c = _case([n, n], [500, 100], 16, 2, d, 32, io, seed=n + d)
    g = np.random.default_rng(n)
    _scale_values(c, lambda s, j: 2.0 ** g.integers(-9, 6, c.hkv))
    _check(c, max_q=n)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("io,e", [(BF, -40), (BF, 40), (FP, -9), (FP, 9)])
def test_scales_far_from_one(n, io, e):
    c = _case([n], [200], 8, 1, 128, 16, io, seed=n)
    _scale_values(c, lambda s, j: np.full(1, 2.0 ** e))
    c.v64 = [v * 2.0 ** -e for v in c.v64]                     # the oracle in units of 2^e

    def scaled(forward):
        def call(**kw):
            out, lse = forward(**kw)
            return out.float() * 2.0 ** -e, lse
        return call

    c.forward = scaled(c.forward)
    _check(c, max_q=n)
