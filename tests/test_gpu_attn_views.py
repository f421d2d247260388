"""Attention operators on arrays that start anywhere: lengths, offsets, tables,
positions, statistics and weights are only as aligned as their elements."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

BF, I8 = torch.bfloat16, torch.int8


def _odd(t):
    """The same values one element past an aligned address."""
    wide = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    at = wide[1:].view(t.shape)
    at.copy_(t)
    assert at.data_ptr() % 16 == t.element_size() and at.is_contiguous()
    return at


@pytest.mark.parametrize("kv", [BF, I8])
@pytest.mark.parametrize("n", [1, 12, 60])
def test_arrays_at_odd_addresses(kv, n):
    # one token, 48 rows and 240 rows per K/V head; sequences that end inside a unit of 64 cells and inside a tile
    from attn_helpers import Case, check_forward, score_error
    from expert_cached_decode_gb300.attention import Rope
    lens = [n + 30, 333, n]
    c = Case([n] * 3, lens, 8, 2, 128, 24, kv, BF, seed=n, rope=Rope(128))
    c.d_cu, c.d_lens, c.d_table = _odd(c.d_cu), _odd(c.d_lens), _odd(c.d_table)
    out = torch.empty((3 * n, 8, 128), dtype=BF, device="cuda")
    lse = _odd(torch.zeros((3 * n, 8), device="cuda"))
    c.att.moe_attn_forward(c.cells, c.q, c.d_cu, c.d_lens, c.d_table, out, lse, max_q=n)
    c.att.moe_attn_sync()
    check_forward(c, out, lse, oa.attention)
    acc = _odd(torch.full((3, 335), 3.0, device="cuda"))
    c.att.moe_attn_weights(c.cells, c.q, lse, c.d_cu, c.d_lens, c.d_table, acc, acc, decay=0.5, max_q=n)
    c.att.moe_attn_sync()
    l64 = lse.double().cpu().numpy()
    for s, length in enumerate(lens):
        w = oa.weights(c.q64[c.rows(s)], c.k64[s], l64[c.rows(s)], 0, c.scale)
        # scores, exponential and fp32 sums of up to 480 rows
        rel = score_error(c, s) + 2.0 ** -19 + 2.0 ** -15
        got = acc[s].double().cpu().numpy()
        assert (np.abs(got[:length] - (w + 1.5)) <= rel * w + 2.0 ** -22 * (w + 1.5)).all()
        assert (got[length:] == 3.0).all()
    # written and read back, at the cells' places and at the same positions given
    k, v = (torch.randn((3 * n, 2, 128), device="cuda").to(BF) for _ in range(2))
    pos = np.concatenate([np.arange(length - n, length) for length in lens]).astype(np.int32)
    c.att.moe_attn_append(c.cells, None, k, v, None, c.d_cu, c.d_lens, c.d_table, None)
    want = c.cells.clone()
    c.att.moe_attn_append(c.cells, None, k, v, _odd(torch.from_numpy(pos).cuda()), c.d_cu, c.d_lens, c.d_table, None)
    assert torch.equal(c.cells, want)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    c.att.moe_attn_read(c.cells, c.d_cu, c.d_lens, c.d_table, ko, vo)
    if kv == BF:
        assert torch.equal(vo, v)
    # an eviction to pages of their own
    budget = 40
    cells = torch.cat([c.cells, torch.zeros((6, 24, c.cb), dtype=torch.uint8, device="cuda")])
    new = _odd(torch.arange(c.n_pages, c.n_pages + 6, dtype=torch.int32, device="cuda").view(3, 2))
    keep = _odd(torch.zeros((3, budget), dtype=torch.int32, device="cuda"))
    new_lens, acc_out = _odd(torch.zeros(3, dtype=torch.int32, device="cuda")), _odd(torch.zeros((3, budget), device="cuda"))
    c.att.moe_attn_evict(cells, acc, c.d_lens, c.d_table, 5, new, keep, new_lens, acc_out)
    c.att.moe_attn_sync()
    a = acc.cpu().numpy()
    for s, length in enumerate(lens):
        kept = oa.evict(a[s, :length], budget, 5)
        assert np.array_equal(keep[s].cpu().numpy()[:len(kept)], kept) and int(new_lens[s]) == len(kept)
        assert np.array_equal(acc_out[s].cpu().numpy()[:len(kept)], a[s][kept])
