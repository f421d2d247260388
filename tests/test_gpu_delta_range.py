"""The gated delta rule over the whole range of fp32: large states and values, and
states far above the values that come to them, in chunks against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from delta_helpers import EPS, Case, unit
from expert_cached_decode_gb300 import GatedDelta
from oracle import delta as od

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def floors(c, s):
    """What the units of a chunk add to Case.check's bounds: out [n, hv, dv], state [hv, dv].

    In chunks the numbers of a column (one of v_dim) are fp16 numbers or pairs of them under one power of two for all tokens,
    which brings a bound B of them to [2^13, 2^14).  fp16 ends at 2^-24, so each is off by 2^-25 2^-13 B at most, however small
    it is.  The bounds, with v the column's largest value in the chunk and s its state's largest number before the chunk:
        Z:  v + L max e^(G_j) S        U:  max_i sum |T_ij| v + L max_i sum |T_ij| e^(G_j) S
        next S:  2.02 (sum_i e^(G_C - G_i) beta_i |k^_i| v + 128^1/2 e^(G_C) s)      (beta_i |k^_i|^2 in [0, 2])
    where S is the bound of the state at hand (s itself before the first chunk), L = 22.63 (the sum of a key's 128 numbers, as
    they are stored: a row shorter than 2)."""
    r = slice(int(c.cu[s]), int(c.cu[s + 1]))
    q, k, v = (x[r] for x in c.views(c.x64))
    g, b = c.g64[r], c.b64[r]
    rep = c.hv // c.hk
    q, k = np.repeat(od.unit(q, EPS), rep, 1), np.repeat(od.unit(k, EPS), rep, 1)
    S = c.st64[c.s_in[s]].copy() if c.s_in[s] >= 0 else np.zeros_like(c.st64[0])
    L, fl = 22.63, 2.0 ** -38
    out, E, B = np.zeros_like(v), np.zeros((c.hv, c.dv)), np.abs(S).max(1)
    for t0 in range(0, len(v), 64):
        w = slice(t0, min(t0 + 64, len(v)))
        top, big, n = np.abs(S).max(1), np.abs(v[w]).max(0), len(v[w])
        for h in range(c.hv):
            G = np.cumsum(g[w, h])
            D = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0.0)))
            K, Q = k[w, h], q[w, h]
            T = np.abs(np.linalg.inv(np.eye(n) + np.tril(b[w, h][:, None] * D * (K @ K.T), -1)) * b[w, h][None])
            P, e, rest = np.abs(D * (Q @ K.T)), np.exp(G), np.exp(G[-1] - G)
            late = T @ e
            bz = big[h] + L * e.max() * B[h]
            bu = T.sum(1).max() * big[h] + L * late.max() * B[h]
            bs = 2.02 * ((rest @ b[w, h]) * big[h] + 11.32 * e[-1] * top[h])
            ez = fl * (11.4 * e[:, None] * B[h] + bz)                     # of Z's tokens, [n, dv]
            eu = T @ ez
            out[w, h] = c.scale * (e[:, None] * (E[h] + fl * 11.4 * B[h]) + P @ (eu + fl * bu))
            E[h] = e[-1] * E[h] + rest @ eu + n * fl * bs
            B[h] = bs
        for t in range(t0, t0 + n):
            S = S * np.exp(g[t])[:, None, None]
            S = S + k[t][:, :, None] * (b[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t])))[:, None, :]
    return out, E


def check(c, d, chunked):
    torch.cuda.synchronize()
    out, state = d["out"].double().cpu().numpy(), d["state"].double().cpu().numpy()
    q, k, v = c.views(c.x64)
    eps, half = 2.0 ** -17, 2.0 ** -10 if chunked else 0.0               # as in Case.check
    for s in range(c.S):
        r = slice(int(c.cu[s]), int(c.cu[s + 1]))
        S0 = c.st64[c.s_in[s]] if c.s_in[s] >= 0 else np.zeros_like(c.st64[0])
        o, S1, mag, size = od.rule(q[r], k[r], v[r], c.g64[r], c.b64[r], S0, c.scale)
        fo, fs = floors(c, s) if chunked else (0.0, 0.0)
        off = np.abs(out[r] - o)
        tol = unit(c.dtype) * 1.01 * np.abs(o) + half * mag + eps * (mag + c.scale * size) + 2.0 ** -24 + fo
        assert (off <= tol).all(), (s, (off / tol).max())
        off = np.sqrt(((state[c.s_out[s]] - S1) ** 2).sum(1))
        assert (off <= eps * size[-1] + 2.0 ** -40 + fs).all(), s


@pytest.mark.parametrize("n", [25, 64, 150, 1600])
@pytest.mark.parametrize("state,value", [(118, 0), (0, 118), (118, 118), (100, 120)])
def test_states_and_values_near_the_end_of_fp32(n, state, value):
    # 2^118 times a few: every sum of the formulas stays below 2^127
    c = Case([n, n], hk=1, hv=2, seed=n, fresh=(1,), dtype=BF)
    c.st64 *= 2.0 ** state
    c.x[:, 2 * c.nq:] *= 2.0 ** value
    c.x64 = c.x.double().cpu().numpy()
    check(c, c.forward(), True)
    check(c, c.forward(max_q=1), False)


@pytest.mark.parametrize("n", [64, 150, 700])
@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_states_far_above_the_values(n, dtype):
    # the state decays to the values' size over some chunks, in every column from another size on
    c = Case([n], hk=1, hv=2, seed=n, dtype=dtype, keep=(0,))
    c.st64 = (c.st64 * 2.0 ** np.linspace(-10, 34 if dtype == BF else 14, 128).round()).astype(np.float32).astype(np.float64)
    check(c, c.forward(), True)


@pytest.mark.parametrize("n", [150, 130])
def test_states_far_above_the_values_without_eps(n):
    # the rows behind a sequence's end have no length: they must not reach the bounds
    c = Case([n], hk=1, hv=2, seed=150, dtype=BF, keep=(0,))
    c.st64 = (c.st64 * 2.0 ** np.linspace(-10, 34, 128).round()).astype(np.float32).astype(np.float64)
    c.op = GatedDelta(1, 2, 128, 128, dtype=BF, eps=0.0)          # (the oracle's eps is 2^-26 of a key's square)
    check(c, c.forward(), True)
    c.b64[:] = 2.0                                                # |k^|^2 is 1 but for its rounding
    c.b64[3] = 0.0
    check(c, c.forward(), True)


def test_columns_of_every_size_next_to_each_other():
    c = Case([100], hk=1, hv=1, seed=2)
    size = 2.0 ** np.linspace(-40, 118, 128).round()
    c.st64 = (c.st64 * size).astype(np.float32).astype(np.float64)
    v = c.x[:, 2 * c.nq:2 * c.nq + 128]
    v.copy_((v.double() * torch.from_numpy(size).cuda()).to(BF))
    c.x64 = c.x.double().cpu().numpy()
    c.check(c.forward())
