"""The gated delta rule as programs use it: tensors side by side in one
allocation, threads, streams, graphs on one handle, and a layer's calls in a row."""

import numpy as np
import pytest
import torch

from delta_helpers import Case

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 4, 128, 128), (2, 2, 128, 64), (1, 1, 64, 128)])
def test_out_directly_behind_or_before_the_inputs(n, hk, hv, dk, dv):
    # rows of q, k, v and out that touch, in either order, are apart: none may count with another's width
    c = Case([n], hk=hk, hv=hv, dk=dk, dv=dv, seed=n)
    q, k, v = (t.contiguous() for t in c.views(c.x))
    for order in ("qkvo", "ovkq", "vokq", "kqov", "vqok"):
        d = c.device()
        t = dict(q=q, k=k, v=v, o=d["out"])
        flat = torch.empty(sum(x.numel() for x in t.values()), dtype=c.dtype, device="cuda")
        at, got = 0, {}
        for name in order:
            got[name] = flat[at:at + t[name].numel()].view(t[name].shape)
            got[name].copy_(t[name])
            at += t[name].numel()
        d["out"] = got["o"]
        c.op.moe_delta_forward(got["q"], got["k"], got["v"], **d)
        c.check(d)
