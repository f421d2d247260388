"""Set-up shared by the tests of the gated delta rule: seeded sequences, slots in
shuffled order, and the checks against the 64-bit oracle."""

import numpy as np
import torch

from expert_cached_decode_gb300 import GatedDelta
from oracle import delta as od

EPS = 1e-6


def unit(dtype):
    """Half a step of a 16-bit type: 2^-8 in bfloat16, 2^-11 in float16 (relative to the value)."""
    return torch.finfo(dtype).eps / 2


class Case:
    """lens[s] tokens per sequence, `pad` rows behind the last one, states in shuffled slots; fresh: sequences that start
    from zeros, drop: that do not keep their state, keep: those whose state goes to another slot."""

    def __init__(self, lens, hk=2, hv=4, dk=128, dv=128, dtype=torch.bfloat16, normalize=True, seed=0, pad=0, fresh=(), drop=(),
                 keep=(), scale=0.0, decay=0.1, gap=8, same_keys=False):
        g = np.random.default_rng(seed)
        self.lens, self.hk, self.hv, self.dk, self.dv, self.dtype = list(lens), hk, hv, dk, dv, dtype
        self.normalize, self.scale = normalize, scale or dk ** -0.5
        S, T = len(lens), int(sum(lens))
        self.S, self.T, self.pad = S, T, pad
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        order = g.permutation(2 * S + 2).astype(np.int32)
        self.n_slots = 2 * S + 2
        self.s_in, self.s_out = order[:S].copy(), order[:S].copy()
        for s in keep:
            self.s_out[s] = order[S + s]
        for s in fresh:
            self.s_in[s] = -1
        for s in drop:
            self.s_out[s] = -1
        nq, nv = hk * dk, hv * dv
        x = g.standard_normal((T + pad, 2 * nq + nv + gap)).astype(np.float32)     # q, k, v: slices of one row
        if same_keys:
            x[:, nq:2 * nq] = x[:1, nq:2 * nq]
        if not normalize:
            qk = x[:, :2 * nq].reshape(T + pad, 2 * hk, dk)
            x[:, :2 * nq] = (qk / np.sqrt((qk * qk).sum(-1, keepdims=True) + EPS)).reshape(T + pad, -1)
        x = torch.from_numpy(x).to(dtype)
        self.x64 = x.double().numpy()
        self.g64 = -(g.random((T + pad, hv)) ** 4 * decay * 10).astype(np.float32).astype(np.float64)
        self.b64 = g.random((T + pad, hv)).astype(np.float32).astype(np.float64)
        self.st64 = (g.standard_normal((self.n_slots, hv, dk, dv)) * 0.3).astype(np.float32).astype(np.float64)
        self.x = x.cuda()
        self.nq = nq
        self.op = GatedDelta(hk, hv, dk, dv, dtype=dtype, normalize=normalize, eps=EPS, scale=scale)

    def views(self, x):
        n, nq = x.shape[0], self.nq
        return (x[:, :nq].reshape(n, self.hk, self.dk) if isinstance(x, np.ndarray) else x[:, :nq].view(n, self.hk, self.dk),
                x[:, nq:2 * nq].reshape(n, self.hk, self.dk) if isinstance(x, np.ndarray) else x[:, nq:2 * nq].view(n, self.hk, self.dk),
                x[:, 2 * nq:2 * nq + self.hv * self.dv].reshape(n, self.hv, self.dv) if isinstance(x, np.ndarray)
                else x[:, 2 * nq:2 * nq + self.hv * self.dv].view(n, self.hv, self.dv))

    def device(self):
        """What a call takes, anew: g, beta, state, out, cu, slots."""
        f = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
        return dict(g=f(self.g64), beta=f(self.b64), state=f(self.st64),
                    out=torch.full((self.T + self.pad, self.hv, self.dv), 7.0, dtype=self.dtype, device="cuda"),
                    cu=torch.from_numpy(self.cu).cuda(), slots_in=torch.from_numpy(self.s_in).cuda(),
                    slots_out=torch.from_numpy(self.s_out).cuda())

    def forward(self, d=None, **kw):
        d = self.device() if d is None else d
        q, k, v = self.views(self.x)
        self.op.moe_delta_forward(q, k, v, **d, **kw)
        return d

    def check(self, d, writes=None, chunked=True):
        """out and state against the oracle; writes: sequences whose state is expected (default: those with a slot)."""
        torch.cuda.synchronize()
        out, state = d["out"].double().cpu().numpy(), d["state"].double().cpu().numpy()
        want = self.st64.copy()
        q, k, v = self.views(self.x64)
        # Sums of up to 128 fp32 terms, and operands that hold 22 bits: 2^-17 of the magnitudes that go into a column.  The
        # rule does not lengthen an error (its steps are contractions), so they add up as `size` does.
        eps = 2.0 ** -17
        # the outputs' own products: operands of 11 bits, two of them a term (token by token: fp32)
        half = 2.0 ** -10 if chunked else 0.0
        for s in range(self.S):
            r = slice(int(self.cu[s]), int(self.cu[s + 1]))
            S0 = self.st64[self.s_in[s]] if self.s_in[s] >= 0 else np.zeros_like(self.st64[0])
            o, S1, mag, size = od.rule(q[r], k[r], v[r], self.g64[r], self.b64[r], S0, self.scale, self.normalize, EPS)
            if self.lens[s]:
                tol = unit(self.dtype) * 1.01 * np.abs(o) + half * mag + eps * (mag + self.scale * size) + 2.0 ** -24
                bad = np.abs(out[r] - o) > tol
                assert not bad.any(), (s, np.argwhere(bad)[:5], np.abs(out[r] - o).max(), tol.max())
            slot = self.s_out[s]
            if slot >= 0 and (writes is None or s in writes):
                off = np.sqrt(((state[slot] - S1) ** 2).sum(1))           # per column
                lim = eps * size[-1] + 2.0 ** -40
                assert (off <= lim).all(), (s, np.argwhere(off > lim)[:5], (off / lim).max())
                want[slot] = state[slot]
        assert np.array_equal(state, want)                               # every other slot as it was
        assert (out[self.T:] == 7.0).all()                               # rows that no sequence holds
