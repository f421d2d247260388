"""Offsets that the gates alone find out of range are reported like those that the
other calls find."""

import pytest
import torch

from expert_cached_decode_gb300 import GatedDelta, MoeError

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_seqs", [1, 40])
def test_gates_alone_report_offsets(n_seqs):
    hv, n = 3, 2 * n_seqs
    op = GatedDelta(1, hv, 64, 64)
    a, b = (torch.randn(n, hv, device="cuda").to(torch.bfloat16) for _ in range(2))
    z = torch.zeros(hv, device="cuda")
    g, beta = (torch.full((n, hv), 7.0, device="cuda") for _ in range(2))
    slots = torch.full((n_seqs,), -1, dtype=torch.int32, device="cuda")
    cu = 2 * torch.arange(n_seqs + 1, dtype=torch.int32, device="cuda")
    call = lambda cu: op.moe_delta_prepare(None, None, None, None, None, a, b, z, z, g, beta, cu, slots, slots)
    call(cu)
    op.moe_delta_sync()                        # nothing is wrong
    want = g.clone()
    bad = cu.clone()
    bad[-1] = n + 5                            # cut to the rows that there are
    g.fill_(7.0)
    call(bad)
    with pytest.raises(MoeError, match="offset"):
        op.moe_delta_sync()
    assert torch.equal(g, want)
    op.moe_delta_sync()                        # once
    slots[0] = 10 ** 9                         # no slot is touched
    call(cu)
    op.moe_delta_sync()
