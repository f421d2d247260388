"""Tokens that no sequence holds (padding after the last offset): their rows are
left as they were, in every kernel."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, I8 = torch.bfloat16, torch.int8


@pytest.mark.parametrize("kv", [BF, I8])
@pytest.mark.parametrize("n", [1, 10, 70])
@pytest.mark.parametrize("max_q", [None, 1])
def test_rows_of_padding_tokens_are_left_alone(kv, n, max_q):
    from attn_helpers import Case
    c = Case([n, n], [n + 200, n + 40], 8, 2, 128, 32, kv, BF, seed=n)
    want, want_l = c.forward(max_q=n)
    acc, acc_want = (torch.zeros((2, n + 200), device="cuda") for _ in range(2))
    args = (c.d_cu, c.d_lens, c.d_table)
    c.att.moe_attn_weights(c.cells, c.q, want_l, *args, None, acc_want, max_q=n)
    q = torch.cat([c.q, torch.full((5, 8, 128), float("nan"), dtype=BF, device="cuda")])
    out, lse = torch.full((2 * n + 5, 8, 128), 7.0, dtype=BF, device="cuda"), torch.full((2 * n + 5, 8), 7.0, device="cuda")
    c.att.moe_attn_forward(c.cells, q, *args, out, lse, max_q=max_q or n)
    c.att.moe_attn_weights(c.cells, q, lse, *args, None, acc, max_q=n)
    c.att.moe_attn_sync()
    assert (out[2 * n:] == 7.0).all() and (lse[2 * n:] == 7.0).all()
    if max_q is None:
        assert torch.equal(out[:2 * n], want) and torch.equal(lse[:2 * n], want_l) and torch.equal(acc, acc_want)
    assert (out[:2 * n].double() - want.double()).abs().max() <= 2.0 ** -6 * want.double().abs().max()
