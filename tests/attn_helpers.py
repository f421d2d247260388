"""Set-up shared by the attention tests: seeded sequences over shuffled pages,
cells in every format, and the same values in 64 bits for the oracle."""

import numpy as np
import torch

from expert_cached_decode_gb300.attention import PagedAttention, kv_cell_bytes

NAN_BYTE = {torch.bfloat16: 0xFF, torch.float16: 0xFF, torch.int8: 0xFF}   # 16-bit NaN; a NaN scale for int8 cells


def quantise(x):
    """int8 codes and fp32 scales of head vectors (numpy, fp32 in)."""
    top = np.abs(x).max(-1, keepdims=True)
    inv = np.where(top > 0, np.float32(127) / np.maximum(top, np.float32(1e-38)), np.float32(0)).astype(np.float32)
    return np.rint(x * inv).astype(np.int8), (top / np.float32(127)).astype(np.float32)


class Case:
    """n_new[s] new tokens and kv_lens[s] cells per sequence.  Cells that no sequence holds, and the rest of each
    sequence's last page, are filled with NaN patterns."""

    def __init__(self, n_new, kv_lens, hq, hkv, d, page, kv_dtype, dtype, window=0, seed=0, pad=0, table_extra=1, scale=0.0,
                 rope=None, std=1.0, q_gap=0):
        g = np.random.default_rng(seed)
        self.n_new, self.kv_lens, self.hq, self.hkv, self.d, self.page = n_new, kv_lens, hq, hkv, d, page
        self.kv_dtype, self.dtype, self.window = kv_dtype, dtype, window
        self.scale = scale or d ** -0.5
        self.cb = kv_cell_bytes(hkv, d, kv_dtype) + pad
        n, need = len(kv_lens), [-(-l // page) for l in kv_lens]
        self.n_pages = sum(need) + 3
        order = g.permutation(self.n_pages)
        self.table = np.zeros((n, max(need) + table_extra), np.int32)
        at = 0
        for s in range(n):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.free = order[at:]
        tokens = int(sum(n_new))
        self.tokens = tokens
        self.cu_q = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        # q as a slice of a wider row: its token stride is not its width
        wide = torch.from_numpy((g.standard_normal((max(tokens, 1), hq + q_gap, d)) * std).astype(np.float32)).to(dtype)
        self.q64 = wide[:tokens, :hq].double().numpy()
        cells = np.full((self.n_pages, page, self.cb), 0xFF, np.uint8)
        self.k64, self.v64 = [], []
        for s in range(n):
            if kv_lens[s] == 0:
                self.k64.append(np.zeros((0, hkv, d)))
                self.v64.append(np.zeros((0, hkv, d)))
                continue
            kv = (g.standard_normal((kv_lens[s], 2, hkv, d)) * std).astype(np.float32)
            if kv_dtype == torch.int8:
                codes, sc = quantise(kv)
                raw = np.concatenate([codes.reshape(kv_lens[s], -1).view(np.uint8),
                                      np.ascontiguousarray(sc).reshape(kv_lens[s], -1).view(np.uint8)], 1)
                val = codes.astype(np.float64) * sc
            else:
                t = torch.from_numpy(kv).to(kv_dtype)
                raw = t.view(torch.int16).numpy().reshape(kv_lens[s], -1).view(np.uint8)
                val = t.double().numpy()
            for j in range(kv_lens[s]):
                cells[self.table[s, j // page], j % page, :raw.shape[1]] = raw[j]
            self.k64.append(val[:, 0])
            self.v64.append(val[:, 1])
        self.cells = torch.from_numpy(cells).cuda()
        self.q = wide.cuda()[:tokens, :hq]
        self.d_cu, self.d_lens = torch.from_numpy(self.cu_q).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
        self.d_table = torch.from_numpy(self.table).cuda()
        self.att = PagedAttention(hq, hkv, d, page, kv_dtype=kv_dtype, dtype=dtype, cell_bytes=self.cb, window=window,
                                  scale=scale, rope=rope)

    def rows(self, s):
        return slice(int(self.cu_q[s]), int(self.cu_q[s + 1]))

    def forward(self, **kw):
        out = torch.full((self.tokens, self.hq, self.d), 7.0, dtype=self.dtype, device="cuda")
        lse = torch.full((self.tokens, self.hq), 7.0, dtype=torch.float32, device="cuda")
        self.att.moe_attn_forward(self.cells, self.q, self.d_cu, self.d_lens, self.d_table, out, lse, **kw)
        torch.cuda.synchronize()
        return out, lse


def unit(dtype):
    """Unit roundoff of a 16-bit type with a significand of p bits, 2^-p: 8 bits in bfloat16, 11 in float16."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11


def score_error(case, s):
    """Bound of the error of a scaled score: fp32 sums of exact products, 2^-20 of the sum of their magnitudes."""
    qa = np.abs(case.q64[case.rows(s)]).max(initial=0.0)
    ka = np.abs(case.k64[s]).max(initial=0.0)
    return 2.0 ** -20 * case.scale * case.d * qa * ka


def check_forward(case, out, lse, oracle_attention):
    got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    p_type = torch.bfloat16 if case.kv_dtype == torch.int8 else case.kv_dtype
    for s in range(len(case.kv_lens)):
        r = case.rows(s)
        want, want_l, mag = oracle_attention(case.q64[r], case.k64[s], case.v64[s], case.window, case.scale)
        es = score_error(case, s)
        empty = np.isneginf(want_l)
        assert np.array_equal(np.isneginf(got_l[r]), empty)
        if empty.any():
            assert not got[r][empty].any()
        ok = ~empty
        if ok.any():
            assert np.abs(got_l[r][ok] - want_l[ok]).max() <= 2 * es + 2.0 ** -21 * np.abs(want_l[ok]).max() + 2.0 ** -20
        # probabilities: rounded to 16 bits (below the fp16 normals: to 2^-25 of the largest), 2 es from the scores;
        # the output: rounded once
        vmax = np.abs(case.v64[s]).max(initial=0.0)
        tiny = 2.0 ** -25 * case.kv_lens[s] * vmax if p_type == torch.float16 else 0.0
        tol = (unit(p_type) * 1.01 + 2 * es + 2.0 ** -18) * mag + tiny + unit(case.dtype) * np.abs(want) * 1.01 + 2.0 ** -24
        bad = np.abs(got[r] - want) > tol
        assert not bad.any(), (s, np.argwhere(bad)[:5], np.abs(got[r] - want).max(), tol.max())
