"""Attention operators at lengths that fill the index ranges: sequences whose
table names one large page again and again, so that a length of 2^27 cells
takes a few megabytes of cells."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

BF, I8 = torch.bfloat16, torch.int8


@pytest.mark.parametrize("n,window", [(1, 4096), (40, 300)])
@pytest.mark.parametrize("kv", [BF, I8])
def test_weights_of_a_window_at_the_end_of_a_very_long_cache(n, window, kv):
    # 32 heads on one K/V head: cells 2^27 before the window, times 32, lie past 32 bits.  One token takes the few-row
    # kernel, 40 the one on tensor memory
    from attn_helpers import Case, score_error
    page, length = 65536, (1 << 27) - 1000
    c = Case([0], [page], 32, 1, 64, page, kv, BF, window=window, seed=n)
    table = torch.full((1, 1 << 11), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    g = np.random.default_rng(n)
    q = torch.from_numpy(g.standard_normal((n, 32, 64)).astype(np.float32)).to(BF).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((n, 32), device="cuda")
    c.att.moe_attn_forward(c.cells, q, cu, lens, table, out, lse, max_q=n)
    acc = torch.full((1, length), 2.0, device="cuda")
    c.att.moe_attn_weights(c.cells, q, lse, cu, lens, table, acc, acc, decay=0.5, max_q=n)
    c.att.moe_attn_sync()
    # the cells that some row sees: the last n - 1 + window
    m = n - 1 + window
    j = np.arange(length - m, length) % page
    c.q64, c.cu_q = q.double().cpu().numpy(), np.array([0, n])
    k, v = c.k64[0][j], c.v64[0][j]
    want, want_l, mag = oa.attention(c.q64, k, v, window, c.scale)
    es = score_error(c, 0)
    got_l = lse.double().cpu().numpy()
    assert np.abs(got_l - want_l).max() <= 2 * es + 2.0 ** -21 * np.abs(want_l).max() + 2.0 ** -20
    # probabilities and output rounded to 16 bits
    assert (np.abs(out.double().cpu().numpy() - want) <= (2.0 ** -8 * 1.01 * 2 + 2 * es + 2.0 ** -18) * mag + 2.0 ** -24).all()
    w = oa.weights(c.q64, k, got_l, window, c.scale)
    got = acc[0, length - m:].double().cpu().numpy()
    # scores and exponentials of a weight, fp32 sums of up to 1,280 rows and of the 1 that was there
    assert (np.abs(got - (w + 1.0)) <= (es + 2.0 ** -19 + 2.0 ** -13) * w + 2.0 ** -22 * (1.0 + w)).all()
    assert (acc[0, :length - m] == 1.0).all()          # the others: the decay alone
    torch.cuda.empty_cache()


def test_an_eviction_whose_budget_fills_the_index_range():
    # the marks behind the kept cells run up to 2^31 - 64 (17 GB of keep and weights)
    from attn_helpers import Case
    c = Case([0], [300], 1, 1, 64, 64, BF, BF)
    budget = 2 ** 31 - 64
    cells = torch.cat([c.cells, torch.zeros((5, 64, c.cb), dtype=torch.uint8, device="cuda")])
    new = torch.full((1, budget // 64), -1, dtype=torch.int32, device="cuda")
    new[0, :5] = torch.arange(c.n_pages, c.n_pages + 5, dtype=torch.int32)
    acc = torch.rand((1, 300), device="cuda")
    keep = torch.full((1, budget), 7, dtype=torch.int32, device="cuda")
    new_lens, acc_out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1, budget), 7.0, device="cuda")
    c.att.moe_attn_evict(cells, acc, c.d_lens, c.d_table, 10, new, keep, new_lens, acc_out)
    c.att.moe_attn_sync()
    assert int(new_lens[0]) == 300
    assert torch.equal(keep[0, :300], torch.arange(300, dtype=torch.int32, device="cuda")) and torch.equal(acc_out[0, :300], acc[0])
    assert int(keep[0, 300:].max()) == -1 == int(keep[0, 300:].min())
    assert float(acc_out[0, 300:].max()) == 0.0 == float(acc_out[0, 300:].min())
    old = c.cells[torch.from_numpy(c.table[0, :5].astype(np.int64)).cuda()].reshape(-1, c.cb)[:300]
    assert torch.equal(cells[c.n_pages:].reshape(-1, c.cb)[:300], old)
    del keep, acc_out, new
    torch.cuda.empty_cache()
