"""Oracle of the attention over a paged cache (test infrastructure only).

Plain numpy in 64 bits, one sequence and one head at a time, from the
definitions: rotation of pairs by an angle, absmax / 127 codes, softmax of
scaled dot products over the visible cells, the weights it gives to a cell,
and the choice of the cells that an eviction keeps.
"""

import numpy as np


def rotate(x, positions, freqs, factor, rot_dim, interleaved):
    """x [T, H, D] with the first rot_dim dimensions turned by positions[t] * freqs[i] radians."""
    x = np.array(x, dtype=np.float64)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)[None]
    c, s = factor * np.cos(ang)[:, None], factor * np.sin(ang)[:, None]
    if interleaved:
        a, b = x[..., 0:rot_dim:2].copy(), x[..., 1:rot_dim:2].copy()
        x[..., 0:rot_dim:2], x[..., 1:rot_dim:2] = a * c - b * s, b * c + a * s
    else:
        h = rot_dim // 2
        a, b = x[..., :h].copy(), x[..., h:rot_dim].copy()
        x[..., :h], x[..., h:rot_dim] = a * c - b * s, b * c + a * s
    return x


def visible(n, length, window):
    """[n, length] bool: which cells each of the n newest tokens sees."""
    p = length - n + np.arange(n)[:, None]
    j = np.arange(length)[None]
    seen = j <= p
    return seen & (j > p - window) if window else seen


def attention(q, k, v, window, scale):
    """q [n, Hq, D], k and v [length, Hkv, D]: out, lse, and sum_j p_j |v_j| (for error bounds)."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    out, bound, lse = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    seen = visible(n, length, window)
    for h in range(hq):
        kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
        for t in range(n):
            at = np.nonzero(seen[t])[0]
            if at.size == 0:
                continue
            x = kh[at] @ q[t, h] * scale
            m = x.max()
            e = np.exp(x - m)
            lse[t, h] = m + np.log(e.sum())
            out[t, h] = e @ vh[at] / e.sum()
            bound[t, h] = e @ np.abs(vh[at]) / e.sum()
    return out, lse, bound


def weights(q, k, lse, window, scale):
    """[length]: what the rows' attention gives to each cell."""
    n, hq, _ = q.shape
    length, hkv, _ = k.shape
    seen = visible(n, length, window)
    total = np.zeros(length)
    for h in range(hq):
        x = q[:, h] @ k[:, h // (hq // hkv)].T * scale
        for t in range(n):
            if np.isfinite(lse[t, h]):
                total[seen[t]] += np.exp(x[t][seen[t]] - lse[t, h])
    return total


def evict(acc, budget, recent):
    """Indices (ascending) of the cells of one sequence that stay; acc [length]."""
    length = len(acc)
    if length <= budget:
        return np.arange(length)
    old = length - min(recent, length)
    rank = [(-(-np.inf if np.isnan(a) else float(a)), j) for j, a in enumerate(acc[:old])]
    chosen = sorted(j for _, j in sorted(rank)[:budget - (length - old)])
    return np.array(chosen + list(range(old, length)), dtype=np.int64)
