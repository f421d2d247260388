"""The gated delta rule's kernels held to the bits that each of them keeps: token
by token everything in fp32; in chunks the state, and for fp16 outputs all but
P's 11 bits."""

import numpy as np
import pytest
import torch

from delta_helpers import EPS, Case, unit
from oracle import delta as od

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
LAYOUTS = [(128, 128, BF), (128, 128, HF), (64, 64, HF), (64, 64, BF), (128, 64, HF), (64, 128, BF)]


# ------------------------------------------------------------ token by token --
# 2^-17 of the magnitudes (Case.check without the chunks' 2^-10): a token's sums take 32 steps one after another and a few more
# across lanes, some 44 2^-24 with the key's norm; the state is rounded twice a token, 24 tokens 2^-18.4 of it; together below 2^-17.
@pytest.mark.parametrize("lens", [[1], [2, 9], [8], [24], [1, 1, 1], [0, 1, 0, 7], [17, 3, 24, 23]])
@pytest.mark.parametrize("dk,dv,dtype", LAYOUTS)
def test_steps(lens, dk, dv, dtype):
    c = Case(lens, dk=dk, dv=dv, dtype=dtype, pad=3, seed=sum(lens))
    c.check(c.forward(max_q=max(lens)), chunked=False)
    c.check(c.forward(), chunked=False)        # the same kernel, whatever the call's bound


@pytest.mark.parametrize("hk,hv", [(1, 1), (3, 3), (1, 5), (16, 32)])
def test_steps_heads(hk, hv):
    c = Case([3, 2], hk=hk, hv=hv, seed=hv)
    c.check(c.forward(max_q=3), chunked=False)


def test_steps_slots_and_gates():
    c = Case([4, 4, 5, 0, 0, 0, 1], fresh=(0, 4), drop=(1, 5), keep=(2, 3), seed=5)
    c.check(c.forward(), chunked=False)
    for g in (0.0, -30.0):
        c.g64[:] = g
        c.check(c.forward(), chunked=False)
    c.g64[2] = -np.inf
    c.b64[:] = 1.0
    c.check(c.forward(), chunked=False)
    c = Case([7, 14], normalize=False, dtype=HF, scale=0.25, seed=2)
    c.check(c.forward(), chunked=False)
    c = Case([9], seed=4, same_keys=True)
    c.g64[:] = 0.0
    c.b64[:] = 1.0
    c.check(c.forward(), chunked=False)


# -------------------------------------------------------------------- chunks --
def _within_chunks(c, s):
    """scale sum_j |e^(G_i - G_j) q^_i.k^_j| |u_j| over the tokens j <= i of i's chunk: what P's terms come to [n, hv, dv]."""
    r = slice(int(c.cu[s]), int(c.cu[s + 1]))
    q, k, v = (x[r] for x in c.views(c.x64))
    g, b = c.g64[r], c.b64[r]
    rep = c.hv // c.hk
    if c.normalize:
        q, k = od.unit(q, EPS), od.unit(k, EPS)
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    S = c.st64[c.s_in[s]].copy() if c.s_in[s] >= 0 else np.zeros_like(c.st64[0])
    u, mag = np.zeros_like(v), np.zeros_like(v)
    for t in range(len(v)):
        S = S * np.exp(g[t])[:, None, None]
        u[t] = b[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[t][:, None, :]
    for t0 in range(0, len(v), 64):
        w = slice(t0, min(t0 + 64, len(v)))
        G = np.cumsum(g[w], 0)
        m = len(G)
        D = np.where(np.tril(np.ones((m, m), bool))[..., None], np.exp(np.minimum(G[:, None] - G[None], 0.0)), 0.0)
        mag[w] = c.scale * np.einsum("ijh,jhv->ihv", np.abs(D * np.einsum("ihd,jhd->ijh", q[w], k[w])), np.abs(u[w]))
    return mag


@pytest.mark.parametrize("lens", [[64], [40, 25], [130, 64, 200]])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_fp16_outputs_of_chunks(lens, dk, dv):
    # the outputs' rounding, 2^-11 of P's terms (its own rounding), and 2^-17 of the magnitudes for everything else: the state and
    # U, pairs of 22 bits under units that are some 2^8 too large
    c = Case(lens, dk=dk, dv=dv, dtype=HF, seed=dk + dv + len(lens))
    d = c.forward()
    torch.cuda.synchronize()
    out = d["out"].double().cpu().numpy()
    q, k, v = c.views(c.x64)
    for s in range(c.S):
        r = slice(int(c.cu[s]), int(c.cu[s + 1]))
        o, _, mag, size = od.rule(q[r], k[r], v[r], c.g64[r], c.b64[r], c.st64[c.s_in[s]], c.scale)
        tol = unit(HF) * 1.01 * np.abs(o) + 2.0 ** -11 * 1.01 * _within_chunks(c, s) + 2.0 ** -17 * (mag + c.scale * size) + 2.0 ** -24
        off = np.abs(out[r] - o)
        assert (off <= tol).all(), (s, (off / tol).max())


# What stands for the state goes into some ten products and factors of 22 bits and more, each off by 2^-22 of its operand at
# most and by chance in sign; U is a difference of parts about twice its size, and T's rows add up to about twice their largest
# number: some 10^1/2 4 2^-22.8 = 2^-19.1 of the state's length.  One operand of 11 bits anywhere: 2^-12.8.
@pytest.mark.parametrize("lens", [[25], [64], [200, 65], [1700]])
@pytest.mark.parametrize("dk,dv,dtype", LAYOUTS)
def test_states_of_chunks(lens, dk, dv, dtype):
    c = Case(lens, hk=1, hv=2, dk=dk, dv=dv, dtype=dtype, seed=sum(lens), decay=0.01)
    d = c.forward()
    torch.cuda.synchronize()
    q, k, v = c.views(c.x64)
    for s in range(c.S):
        r = slice(int(c.cu[s]), int(c.cu[s + 1]))
        _, want, _, _ = od.rule(q[r], k[r], v[r], c.g64[r], c.b64[r], c.st64[c.s_in[s]], c.scale)
        got = d["state"][int(c.s_out[s])].double().cpu().numpy()
        off = np.sqrt(((got - want) ** 2).sum((1, 2)) / (want ** 2).sum((1, 2)))
        assert (off <= 2.0 ** -17).all(), off
