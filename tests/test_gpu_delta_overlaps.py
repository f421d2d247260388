"""Tensors that share memory with what a call writes are refused by name of the
call; those that lie between the rows of another one are not."""

import pytest
import torch

from delta_helpers import Case
from expert_cached_decode_gb300 import GatedDelta, MoeError, moe_norm_block

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _within(big, like):
    """A tensor like `like` in the memory of `big`."""
    flat = big.view(-1).view(torch.uint8)[:like.numel() * like.element_size()]
    return flat.view(like.dtype).view(like.shape)


def test_forward():
    c = Case([4, 2], seed=1)
    q, k, v = (t.contiguous() for t in c.views(c.x))
    d = c.device()
    small = dict(g=d["g"], beta=d["beta"], cu=d["cu"], slots_in=d["slots_in"], slots_out=d["slots_out"])
    for name, t in small.items():                      # each in the state's memory, then in the output's
        for big in ("state", "out"):
            with pytest.raises(MoeError, match="overlaps"):
                c.op.moe_delta_forward(q, k, v, **{**d, name: _within(d[big], t)})
    for i in range(3):
        t = [q, k, v]
        t[i] = _within(d["state"], t[i])
        with pytest.raises(MoeError, match="overlaps"):
            c.op.moe_delta_forward(*t, **d)
    with pytest.raises(MoeError, match="overlaps"):
        c.op.moe_delta_forward(q, k, v, **{**d, "out": _within(d["state"], d["out"])})
    c.forward(d)                                       # nothing was written so far
    c.check(d)


def test_prepare():
    op = GatedDelta(1, 2, 64, 64, taps=3)
    n, C, r = 8, op.channels, lambda *s: torch.randn(*s, device="cuda").to(BF)
    f = lambda *s: torch.randn(*s, device="cuda")
    d = dict(x=r(n, C), conv_w=r(C, 3), conv_bias=r(C), conv_state=r(9, 2, C), y=r(n, C), a=r(n, 2), b=r(n, 2), a_log=f(2),
             dt_bias=f(2), g=f(n, 2), beta=f(n, 2), cu=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
             slots_in=torch.zeros(1, dtype=torch.int32, device="cuda"), slots_out=torch.zeros(1, dtype=torch.int32, device="cuda"))
    before = {k: t.clone() for k, t in d.items()}
    for name in d:
        for big in ("y", "conv_state"):
            if name != big and not (name == "conv_state" and big == "y"):
                with pytest.raises(MoeError, match="overlaps"):
                    op.moe_delta_prepare(**{**d, name: _within(d[big], d[name])})
    for name in ("a_log", "dt_bias", "cu", "slots_in", "slots_out", "beta"):
        with pytest.raises(MoeError, match="overlaps"):
            op.moe_delta_prepare(**{**d, name: _within(d["g"], d[name])})
    with pytest.raises(MoeError, match="overlaps"):
        op.moe_delta_prepare(**{**d, "a": _within(d["g"], d["a"]), "b": _within(d["g"], d["b"])})
    torch.cuda.synchronize()
    assert all(torch.equal(before[k], d[k]) for k in d)
    op.moe_delta_prepare(**d)
    op.moe_delta_sync()


@pytest.mark.parametrize("n", [3, 40])
def test_between_the_rows(n):
    # rows of q, k, v far apart, the output in the gap behind the first row
    c = Case([n], hk=1, hv=2, seed=n)
    wide = c.x.shape[1] + n * 2 * 128
    wide += -wide % 8
    buf = torch.zeros(n, wide, dtype=BF, device="cuda")
    x = buf[:, :c.x.shape[1]]
    x.copy_(c.x)
    d = c.device()
    d["out"] = buf[0, c.x.shape[1]:c.x.shape[1] + n * 2 * 128].view(n, 2, 128)
    c.op.moe_delta_forward(*c.views(x), **d)
    c.check(d)
    h = torch.randn(n, 64, device="cuda").to(BF)
    y = buf[:, :64]
    w = torch.ones(64, dtype=BF, device="cuda")
    out = buf[0, 64:64 + n * 64].view(n, 64) if n * 64 + 64 <= wide else None
    if out is not None:
        want, y0 = torch.empty_like(h), y.clone()
        moe_norm_block(y0, h, want)
        moe_norm_block(y, h, out)
        assert torch.equal(out, want)
