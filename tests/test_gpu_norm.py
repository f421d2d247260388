"""The norms around the blocks on the GPU against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from delta_helpers import unit
from expert_cached_decode_gb300 import MoeError, moe_norm_block, moe_norm_gated
from oracle import delta as od

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6
# fp32 inside: sums of squares of up to 16,384 terms in 2^9 or fewer steps one after another, a fast exponential and a few
# products: 2^-19 of the result (and of the parts of a sum), on top of the one rounding
IN = 2.0 ** -19


def _t(g, *s, dtype=BF, std=1.0):
    return torch.from_numpy((g.standard_normal(s) * std).astype(np.float32)).to(dtype).cuda()


def _f(t):
    return None if t is None else t.double().cpu().numpy()


def _block(rows, d, io=BF, y=F, h=BF, gate=None, act="sigmoid", post=False, pre=True, scale=1.0, off=0.0, seed=0, gap=0, inplace=False,
           out=True):
    g = np.random.default_rng(seed)
    yt, ht = _t(g, rows, d + gap, dtype=y)[:, :d], None if h is None else _t(g, rows, d + (0 if inplace else gap), dtype=h, std=2)[:, :d]
    gt = {None: None, "token": _t(g, rows, 1, dtype=io), "full": _t(g, rows, d + gap, dtype=io)[:, :d], "column": _t(g, rows, 8, dtype=io)[:, 3:4]}[gate]
    pw, qw = _t(g, d, dtype=io) if post else None, _t(g, d, dtype=io) if pre else None
    want, wx = od.norm_block(_f(yt), _f(ht), _f(gt), _f(pw), _f(qw), act, scale, EPS, off)
    mag = np.abs(want) if ht is None else np.abs(_f(ht)) + np.abs(want - _f(ht))
    dt = h if h is not None else io
    ho = (ht if inplace else torch.full((rows, d), 7.0, dtype=dt, device="cuda")) if out else None
    x = torch.full((rows, d), 7.0, dtype=io, device="cuda") if pre else None
    moe_norm_block(yt, ht, ho, x, pre_w=qw, post_w=pw, gate=gt, act=act, scale=scale, eps=EPS, weight_offset=off)
    torch.cuda.synchronize()
    if out:
        u = unit(dt) if dt != F else 2.0 ** -24
        assert (np.abs(_f(ho) - want) <= (u * 1.01) * np.abs(want) + IN * mag + 2.0 ** -24).all()
    if pre:
        # the sum's own error (IN of its parts), through the norm
        part = IN * mag / np.sqrt((want ** 2).mean(-1, keepdims=True) + EPS) * np.abs(_f(qw) + off)
        assert (np.abs(_f(x) - wx) <= (unit(io) * 1.01 + IN) * np.abs(wx) + part + 2.0 ** -24).all()


@pytest.mark.parametrize("d", [8, 16, 24, 64, 104, 128, 256, 264, 1000, 2048, 2056, 4096, 8192, 9000, 16384])
@pytest.mark.parametrize("rows", [1, 5])
def test_block_lengths(d, rows):
    _block(rows, d, seed=d)
    _block(rows, d, io=HF, y=HF, h=F, gate="full", post=True, scale=0.5, off=1.0, gap=8, seed=d)


@pytest.mark.parametrize("io", [BF, HF])
@pytest.mark.parametrize("y", [F, "io"])
@pytest.mark.parametrize("h", [F, "io", None])
@pytest.mark.parametrize("gate,act,post,pre", [(None, "none", False, True), ("token", "sigmoid", True, True), ("full", "silu", True, False),
                                               ("column", "none", False, True)])
def test_block_parts(io, y, h, gate, act, post, pre):
    k = lambda t: io if t == "io" else t
    _block(37, 520, io=io, y=k(y), h=k(h), gate=gate, act=act, post=post, pre=pre, scale=-0.7, gap=16, seed=1)


def test_block_in_place_and_without_sum():
    _block(9, 2048, inplace=True)
    _block(9, 2048, h=F, y=BF, inplace=True, post=True)
    _block(9, 2048, out=False)
    _block(2000, 2048, seed=2)


def test_block_zero_rows_and_values():
    z = torch.zeros(3, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    h, x = torch.full_like(z, 7.0), torch.full_like(z, 7.0)
    moe_norm_block(z, z, h, x, pre_w=w, post_w=w)
    assert not h.any() and not x.any()
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    moe_norm_block(e, e, e, e, pre_w=w)
    moe_norm_gated(e.view(0, 1, 64), e.view(0, 1, 64), w, e.view(0, 1, 64))
    # rows are apart
    y = torch.randn(4, 2048, device="cuda")
    y[1, 5] = float("nan")
    y[2, 7] = float("inf")
    w = torch.ones(2048, dtype=BF, device="cuda")
    h, x = torch.empty(4, 2048, device="cuda"), torch.empty(4, 2048, dtype=BF, device="cuda")
    moe_norm_block(y, None, h, x, pre_w=w, post_w=w)
    assert torch.isnan(x[1]).all() and torch.isfinite(x[0]).all() and torch.isfinite(x[3]).all()


@pytest.mark.parametrize("d", [8, 64, 72, 128, 256, 512, 2048, 16384])
@pytest.mark.parametrize("act,first", [("silu", False), ("sigmoid", True), ("none", False)])
@pytest.mark.parametrize("io", [BF, HF])
def test_gated(d, act, first, io):
    g = np.random.default_rng(d)
    n, h = 5, 3
    o, z, w = _t(g, n, h + 1, d, dtype=io)[:, :h], _t(g, n, h + 2, d, dtype=io)[:, 2:], _t(g, d, dtype=io)
    out = torch.full((n, h, d), 7.0, dtype=io, device="cuda")
    moe_norm_gated(o, z, w, out, act=act, gate_first=first, eps=EPS, weight_offset=0.5)
    want = od.norm_gated(_f(o), _f(z), _f(w), act, first, EPS, 0.5)
    assert (np.abs(_f(out) - want) <= (unit(io) * 1.01 + IN) * np.abs(want) + 2.0 ** -24).all()
    o = o.contiguous()
    moe_norm_gated(o, z, w, o, act=act, gate_first=first, eps=EPS, weight_offset=0.5)     # in place
    assert torch.equal(o, out)


def test_gated_many_heads():
    g = np.random.default_rng(1)
    o, z, w = _t(g, 301, 32, 128), _t(g, 301, 32, 128), _t(g, 128)
    out = torch.empty_like(o)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    moe_norm_gated(o, z, w, out, stream=s)
    s.synchronize()
    want = od.norm_gated(_f(o), _f(z), _f(w), "silu", False, EPS, 0.0)
    assert (np.abs(_f(out) - want) <= (unit(BF) * 1.01 + IN) * np.abs(want) + 2.0 ** -24).all()


def test_refusals():
    y = torch.zeros(4, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    o = torch.empty_like(y)
    for exc, words, kw in [
            (ValueError, "h must", dict(h=y[:3])), (ValueError, "h_out must", dict(h_out=o[:, :32])), (ValueError, "pre_w must", dict(pre_w=w.float())),
            (ValueError, "x must", dict(x=o.float())), (ValueError, "gate must", dict(gate=y[:, :8])), (ValueError, "y must", dict(y=y.half(), x=None, pre_w=w, h=y)),
            (MoeError, "go together", dict(x=None)), (MoeError, "neither", dict(x=None, pre_w=None, h_out=None)),
            (MoeError, "scale", dict(scale=float("inf"))), (MoeError, "eps", dict(eps=-1.0)), (MoeError, "weight_offset", dict(weight_offset=float("nan"))),
            (KeyError, "tanh", dict(act="tanh"))]:
        with pytest.raises(exc, match=words):
            moe_norm_block(**{**dict(y=y, h=y, h_out=o, x=o, pre_w=w), **kw})
    wide = torch.zeros(4, 68, dtype=BF, device="cuda")
    with pytest.raises(MoeError, match="16-byte"):
        moe_norm_block(wide[:, 4:], y, o, o, pre_w=w)
    with pytest.raises(MoeError, match="multiple of 8"):
        moe_norm_block(torch.zeros(4, 60, dtype=BF, device="cuda"), None, torch.zeros(4, 60, dtype=BF, device="cuda"))
    with pytest.raises(MoeError, match="contiguous"):
        big = torch.zeros(4, 2, 64, dtype=BF, device="cuda")
        moe_norm_gated(big[:, :1], big[:, :1], w, big.view(8, 1, 64)[:4])
    torch.cuda.synchronize()
