"""Gated delta rule, the convolution and gates in front of it, and the norms
around the blocks: plain 64-bit numpy, token by token."""

import numpy as np


def unit(x, eps):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + eps)


def rule(q, k, v, g, beta, state, scale, normalize=True, eps=1e-6):
    """One sequence: q, k [n, hk, dk], v [n, hv, dv], g, beta [n, hv], state [hv, dk, dv].  Returns the outputs [n, hv, dv],
    the new state, and two bounds for error estimates: `mag` [n, hv, dv], the output with every term's magnitude
    (scale * sum over tokens and dimensions of |q^| |k^| |u|, decayed), and `size` [n, hv, dv], the magnitudes that went into
    each column of the state (its 2-norm before, and |u|'s parts with the length of their keys, decayed); size[-1] is that of
    the new state, its first row that of the given one where there are no tokens."""
    n, hv, dv = v.shape
    rep = hv // k.shape[1]
    if normalize:
        q, k = unit(q, eps), unit(k, eps)
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    S = state.copy()
    A = np.abs(S)
    N = np.sqrt((S * S).sum(1))
    out, mag, size = np.zeros((n, hv, dv)), np.zeros((n, hv, dv)), np.zeros((n, hv, dv))
    for t in range(n):
        d = np.exp(g[t])[:, None, None]
        S = S * d
        A = A * d
        seen = np.einsum("hkv,hk->hv", S, k[t])
        u = beta[t][:, None] * (v[t] - seen)
        parts = beta[t][:, None] * (np.abs(v[t]) + np.einsum("hkv,hk->hv", np.abs(S), np.abs(k[t])))
        N = N * d[:, :, 0] + np.sqrt((k[t] ** 2).sum(-1))[:, None] * parts
        S = S + k[t][:, :, None] * u[:, None, :]
        A = A + np.abs(k[t])[:, :, None] * np.abs(u)[:, None, :]
        out[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        mag[t] = scale * np.einsum("hkv,hk->hv", A, np.abs(q[t]))
        size[t] = N
    return out, S, mag, size if n else N[None]


def conv(x, w, bias, old):
    """x [n, C], w [C, taps], bias [C] or None, old [taps - 1, C] inputs before: silu of the convolution, the new `old`, and
    the sums' magnitudes."""
    taps = w.shape[1]
    both = np.concatenate([old, x])
    y, mag = np.zeros_like(x), np.zeros_like(x)
    for i in range(taps):
        y += w[:, i] * both[i:i + len(x)]
        mag += np.abs(w[:, i] * both[i:i + len(x)])
    if bias is not None:
        y += bias
        mag += np.abs(bias)
    return y / (1 + np.exp(-y)), both[len(x):], mag


def gates(a, b, a_log, dt_bias):
    return -np.exp(a_log) * np.logaddexp(0, a + dt_bias), 1 / (1 + np.exp(-b))


def act(z, kind):
    s = 1 / (1 + np.exp(-z))
    return {"none": z, "sigmoid": s, "silu": z * s}[kind]


def rms(x, w, offset, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + offset)


def norm_block(y, h, gate, post_w, pre_w, kind, scale, eps, offset):
    if post_w is not None:
        y = rms(y, post_w, offset, eps)
    if gate is not None:
        y = y * act(gate, kind)
    out = scale * y if h is None else h + scale * y
    return out, None if pre_w is None else rms(out, pre_w, offset, eps)


def norm_gated(o, z, w, kind, gate_first, eps, offset):
    return rms(o * act(z, kind), w, offset, eps) if gate_first else rms(o, w, offset, eps) * act(z, kind)
