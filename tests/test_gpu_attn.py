"""GPU parity of the attention over a paged cache (moe_attn_*) against the
64-bit oracle: cell formats, head layouts, lengths, windows, rows that see
nothing, pages that end inside a tile, NaN in cells that nobody sees, strides,
streams, and values out of range on the GPU."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

BF, FP, I8 = torch.bfloat16, torch.float16, torch.int8


def _case(*a, **k):
    from attn_helpers import Case
    return Case(*a, **k)


def _check(case, **kw):
    from attn_helpers import check_forward
    out, lse = case.forward(**kw)
    case.att.moe_attn_sync()
    check_forward(case, out, lse, oa.attention)
    return out, lse


# --- forward ----------------------------------------------------------------------
@pytest.mark.parametrize("kv,io", [(BF, BF), (FP, FP), (I8, BF), (I8, FP)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (6, 1), (32, 4)])
def test_single_tokens(kv, io, d, hq, hkv):
    lens = [1, 2, 17, 63, 64, 65, 200, 333]
    _check(_case([1] * len(lens), lens, hq, hkv, d, 16, kv, io, seed=hq + d), max_q=1)


@pytest.mark.parametrize("kv,io", [(BF, BF), (FP, FP), (I8, BF), (I8, FP)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (16, 2), (12, 2)])
def test_chunks(kv, io, d, hq, hkv):
    n, lens = [130, 5, 1, 33, 129], [130, 260, 300, 33, 517]
    _check(_case(n, lens, hq, hkv, d, 32, kv, io, seed=hq + d, q_gap=2))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 128, 512])
@pytest.mark.parametrize("n,kv", [(1, BF), (20, BF), (1, I8), (20, I8)])
def test_page_sizes(page, n, kv):
    _check(_case([n, n, n], [n, 150, 301], 8, 2, 128, page, kv, BF, seed=page), max_q=n)


@pytest.mark.parametrize("window", [1, 2, 7, 64, 100, 1000])
@pytest.mark.parametrize("n", [1, 3, 150])
@pytest.mark.parametrize("kv", [FP, I8])
def test_windows(window, n, kv):
    _check(_case([n, n], [n, 420], 8, 4, 64, 16, kv, FP, window=window, seed=window), max_q=n)


@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("kv", [BF, I8])
def test_rows_that_see_nothing(n, kv):
    # more new tokens than cells, no cells at all, no new tokens
    n_new, lens = [n, n, 0, n, n + 6, 0], [0, 1, 50, 90, 3, 0]
    c = _case(n_new, lens, 8, 2, 128, 16, kv, BF, seed=n)
    out, lse = _check(c, max_q=n + 6)
    assert torch.isneginf(lse[:n]).all()


@pytest.mark.parametrize("n,max_q", [(1, 1), (4, 4), (9, 1), (64, 2), (64, 64)])
def test_the_token_hint_changes_no_result_beyond_rounding(n, max_q):
    # max_q only chooses the kernel; a wrong one is no error
    _check(_case([n, 1], [200, 77], 8, 2, 128, 16, BF, BF, seed=n), max_q=max_q)


@pytest.mark.parametrize("kv,n,hq,hkv,d", [(BF, 1, 8, 2, 128), (I8, 1, 8, 1, 128), (I8, 5, 8, 1, 64), (FP, 3, 4, 1, 64),
                                            (BF, 17, 8, 1, 128)])
def test_a_cache_split_over_the_gpu(kv, n, hq, hkv, d):
    io = FP if kv == FP else BF
    c = _case([n, n], [20011, 4099], hq, hkv, d, 64, kv, io, seed=3)
    out, lse = _check(c, max_q=n)
    again, lse2 = c.forward(max_q=n)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_many_sequences_of_uneven_length():
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(0, 400, 333)]
    _check(_case([1] * 333, lens, 4, 1, 64, 16, BF, BF, seed=4), max_q=1)
    _check(_case([int(min(x, l)) for x, l in zip(g.integers(0, 40, 60), lens)], lens[:60], 16, 2, 128, 16, I8, BF, seed=5))


def test_large_scores_and_a_wide_cell():
    # probabilities that are 0 or 1 in effect; cells with space after their data
    _check(_case([1, 70], [300, 300], 8, 2, 128, 16, BF, BF, seed=6, std=6.0, pad=48))
    _check(_case([1, 70], [300, 300], 8, 2, 128, 16, I8, BF, seed=7, std=6.0, pad=16, scale=0.3))


def test_infinite_key_of_a_hidden_cell_reaches_no_row():
    # K of the newest cell is infinite and its V zero: every row but the last has it masked
    for n in (6, 40):
        c = _case([n], [200], 4, 1, 64, 16, BF, BF, seed=8)
        cell = c.cells.view(BF)[c.table[0, 199 // 16], 199 % 16]
        cell[:64] = float("inf")
        cell[64:128] = 0.0
        out, lse = c.forward(max_q=n)
        want, want_l, mag = oa.attention(c.q64[:-1], c.k64[0][:199], c.v64[0][:199], 0, c.scale)
        got = out[:-1].double().cpu().numpy()
        assert np.isfinite(got).all()
        assert np.abs(got - want).max() <= 2.0 ** -7 * mag.max()


def test_empty_calls_and_lse_left_out():
    c = _case([1, 2], [40, 50], 4, 2, 64, 16, BF, BF)
    out, _ = c.forward()
    out2 = torch.zeros_like(out)
    c.att.moe_attn_forward(c.cells, c.q, c.d_cu, c.d_lens, c.d_table, out2)
    assert torch.equal(out, out2)
    z = torch.zeros((0, 4, 64), dtype=BF, device="cuda")
    c.att.moe_attn_forward(c.cells, z, torch.zeros(3, dtype=torch.int32, device="cuda"), c.d_lens, c.d_table, z)
    c.att.moe_attn_forward(c.cells, z, torch.zeros(1, dtype=torch.int32, device="cuda"), c.d_lens[:0], c.d_table[:0], z)
    c.att.moe_attn_sync()


def test_another_stream_and_a_graph():
    c = _case([3, 1], [700, 50], 8, 2, 128, 16, I8, BF, seed=9)
    want, want_l = c.forward(max_q=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.zeros_like(want), torch.zeros_like(want_l)
    c.att.moe_attn_forward(c.cells, c.q, c.d_cu, c.d_lens, c.d_table, out, lse, max_q=3, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.att.moe_attn_forward(c.cells, c.q, c.d_cu, c.d_lens, c.d_table, out, lse, max_q=3)
    out.zero_()
    c.d_lens.copy_(torch.tensor([690, 41], dtype=torch.int32))   # shorter sequences, read when the graph runs
    g.replay()
    torch.cuda.synchronize()
    again, _ = c.forward(max_q=3)
    assert torch.equal(out, again) and not torch.equal(out, want)


def test_values_out_of_range_on_the_gpu_are_reported_and_left_out():
    from expert_cached_decode_gb300 import MoeError
    for n in (1, 40):
        c = _case([n, n], [100, 80], 4, 2, 64, 16, BF, BF, seed=10)
        want, _ = c.forward(max_q=n)
        c.att.moe_attn_sync()
        c.d_table[1, 2] = c.n_pages          # cells 32..47 of sequence 1 are nowhere
        out, lse = c.forward(max_q=n)
        with pytest.raises(MoeError, match="page id"):
            c.att.moe_attn_sync()
        c.att.moe_attn_sync()
        assert torch.equal(out[:n], want[:n])
        at = np.r_[0:32, 48:80]
        if n == 1:
            w, _, mag = oa.attention(c.q64[1:], c.k64[1][at], c.v64[1][at], 0, c.scale)
            assert np.abs(out[1:].double().cpu().numpy() - w).max() <= 2.0 ** -7 * mag.max()
        c.d_table[1, 2] = -1
        c.forward(max_q=n)
        with pytest.raises(MoeError, match="page id"):
            c.att.moe_attn_sync()
        c.d_lens[0] = 10 ** 6                # beyond the table's row
        c.d_table[1, 2] = 0
        c.forward(max_q=n)
        with pytest.raises(MoeError, match="length"):
            c.att.moe_attn_sync()


# --- rotation, cells ----------------------------------------------------------------
def _radians(rot, base, scaling, factor, original_len):
    i = np.arange(rot // 2)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f /= factor
    if scaling == "yarn":
        dim = lambda t: rot * np.log(original_len / (t * 2 * np.pi)) / (2 * np.log(base))
        lo, hi = max(0, np.floor(dim(32.0))), min(rot - 1, np.ceil(dim(1.0)))
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * np.log(factor) + 1
    return f, 1.0


@pytest.mark.parametrize("kv,io", [(BF, BF), (FP, FP), (I8, BF), (I8, FP)])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_append_and_read(kv, io, d, rot, interleaved, scaling):
    from attn_helpers import unit
    from expert_cached_decode_gb300.attention import Rope
    hq, hkv, n, lens = 6, 3, [1, 7, 0, 4], [40, 7, 10, 2]      # the last: more tokens than cells
    rope = Rope(rot, base=5e5, interleaved=interleaved, scaling=scaling, factor=8.0, original_len=8192)
    c = _case(n, lens, hq, hkv, d, 5, kv, io, seed=d + rot, rope=rope)
    g = np.random.default_rng(1)
    qkv = torch.from_numpy(g.standard_normal((12, hq + 2 * hkv, d)).astype(np.float32)).to(io).cuda()
    qkv[3, hq:hq + 1] = 0                                      # a zero head vector
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    pos = torch.tensor([131071, 5, 0, -3, 2 ** 31 - 1, 77, 4096, 1, 9, 12345678, 2, 3], dtype=torch.int32, device="cuda")
    q_out = torch.zeros((12, hq, d), dtype=io, device="cuda")
    before = c.cells.clone()
    c.att.moe_attn_append(c.cells, q, k, v, pos, c.d_cu, c.d_lens, c.d_table, q_out)
    k_out, v_out = (torch.full((12, hkv, d), 7.0, dtype=io, device="cuda") for _ in range(2))
    c.att.moe_attn_read(c.cells, c.d_cu, c.d_lens, c.d_table, k_out, v_out)
    c.att.moe_attn_sync()
    f, factor = _radians(rot, 5e5, scaling, 8.0, 8192) if rot else (np.zeros(0), 1.0)
    q64, k64, v64 = (x.double().cpu().numpy() for x in (q, k, v))
    # the angle: 2^-32 turns and fp32 sine and cosine (2^-21 in all); the result: one rounding.  The reference's own
    # angle is off by 2^31 * 2^-53 radians at the largest position
    for got, want, src in ((q_out, oa.rotate(q64, pos.cpu(), f, factor, rot, interleaved), q64),):
        tol = unit(io) * 1.01 * np.abs(want) + 2.0 ** -19 * np.abs(src).max() * factor + 2.0 ** -24
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    has_cell = np.array([True] * 8 + [False, False, True, True])
    for got, want in ((k_out, oa.rotate(k64, pos.cpu(), f, factor, rot, interleaved)), (v_out, v64)):
        got = got.double().cpu().numpy()
        assert (got[~has_cell] == 7.0).all()
        tol = unit(io) * 1.01 * np.abs(want) + 2.0 ** -19 * np.abs(want).max() + 2.0 ** -24
        if kv == I8:   # half a code, and the read's own rounding
            tol = tol + np.abs(want).max(-1, keepdims=True) / 127 * 0.501 + unit(io) * 1.01 * np.abs(want).max(-1, keepdims=True)
        assert (np.abs(got - want) <= tol)[has_cell].all()
    if kv != I8:
        assert torch.equal(v_out[torch.from_numpy(has_cell).cuda()], v[torch.from_numpy(has_cell).cuda()])
    # nothing else moved: every other cell keeps its bytes
    touched = np.zeros((c.n_pages, 5), bool)
    for s in range(4):
        for i in range(n[s]):
            j = lens[s] - n[s] + i
            if j >= 0:
                touched[c.table[s, j // 5], j % 5] = True
    keep = torch.from_numpy(~touched).cuda()
    assert torch.equal(c.cells[keep], before[keep])


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_frequencies(scaling):
    from expert_cached_decode_gb300.attention import Rope
    r = Rope(64, base=1e6, scaling=scaling, factor=4.0, original_len=32768)
    f, factor = _radians(64, 1e6, scaling, 4.0, 32768)
    assert abs(r.factor - factor) < 1e-12
    assert np.abs(r.turns.astype(np.float64) * 2.0 ** -64 - f / (2 * np.pi)).max() < 2.0 ** -50


def test_append_in_place_alone_and_at_the_cells_places():
    from expert_cached_decode_gb300.attention import Rope
    rope = Rope(128)
    c = _case([3, 2], [9, 20], 4, 2, 128, 16, BF, BF, rope=rope)
    q = c.q.contiguous()
    want = torch.zeros_like(q)
    pos = torch.tensor([6, 7, 8, 18, 19], dtype=torch.int32, device="cuda")
    cells = c.cells.clone()
    c.att.moe_attn_append(c.cells, q, None, None, pos, c.d_cu, c.d_lens, c.d_table, want)
    assert torch.equal(c.cells.view(torch.int16), cells.view(torch.int16))     # only q
    same = q.clone()
    c.att.moe_attn_append(c.cells, same, None, None, None, c.d_cu, c.d_lens, c.d_table, same)
    assert torch.equal(same, want)


@pytest.mark.parametrize("kv,io", [(BF, BF), (I8, BF), (FP, FP)])
def test_what_was_appended_is_what_attention_reads(kv, io):
    # tokens written one call at a time and as one chunk give the same cells and the same attention
    c = _case([12], [12], 8, 2, 128, 4, kv, io, seed=2)
    g = np.random.default_rng(3)
    k, v = (torch.from_numpy(g.standard_normal((12, 2, 128)).astype(np.float32)).to(io).cuda() for _ in range(2))
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    c.cells.zero_()
    for t in range(12):
        c.att.moe_attn_append(c.cells, None, k[t:t + 1], v[t:t + 1], None, one,
                              torch.tensor([t + 1], dtype=torch.int32, device="cuda"), c.d_table, None)
    single = c.cells.clone()
    c.cells.zero_()
    c.att.moe_attn_append(c.cells, None, k, v, None, c.d_cu, c.d_lens, c.d_table, None)
    assert torch.equal(c.cells, single)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    c.att.moe_attn_read(c.cells, c.d_cu, c.d_lens, c.d_table, ko, vo)
    out, lse = c.forward()
    # int8: the values attention uses are the codes times the scale, read back rounded once more
    want, _, mag = oa.attention(c.q64, ko.double().cpu().numpy(), vo.double().cpu().numpy(), 0, c.scale)
    assert np.abs(out.double().cpu().numpy() - want).max() <= (2.0 ** -5 if kv == I8 else 2.0 ** -7) * mag.max()


# --- weights --------------------------------------------------------------------------
@pytest.mark.parametrize("kv,io", [(BF, BF), (FP, FP), (I8, BF), (I8, FP)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n", [(4, 4, [1, 1, 1, 1, 1]), (12, 2, [1, 0, 5, 40, 3]), (16, 2, [3, 33, 130, 7, 12])])
@pytest.mark.parametrize("window", [0, 50])
def test_weights(kv, io, d, hq, hkv, n, window):
    from attn_helpers import score_error
    lens = [129, 40, 300, 40, 2]
    c = _case(n, lens, hq, hkv, d, 24, kv, io, window=window, seed=d + hq)
    _, lse = c.forward()
    g = np.random.default_rng(0)
    acc = torch.from_numpy(g.random((5, 310)).astype(np.float32)).cuda()
    out = torch.full_like(acc, 7.0)
    args = (c.cells, c.q, lse, c.d_cu, c.d_lens, c.d_table)
    c.att.moe_attn_weights(*args, acc, out, decay=0.75)
    zero = torch.full_like(acc, 7.0)
    c.att.moe_attn_weights(*args, None, zero, max_q=max(n))
    inplace = acc.clone()
    c.att.moe_attn_weights(*args, inplace, inplace, decay=0.75)
    c.att.moe_attn_sync()
    assert torch.equal(inplace[:, :300] * 1, torch.where(out[:, :300] == 7.0, acc[:, :300], out[:, :300]))
    l64 = lse.double().cpu().numpy()
    for s in range(5):
        w = oa.weights(c.q64[c.rows(s)], c.k64[s], l64[c.rows(s)], window, c.scale)
        got, got0 = out[s].double().cpu().numpy(), zero[s].double().cpu().numpy()
        # scores, exponential and fp32 sums of up to 130 * 16 rows
        rel = score_error(c, s) + 2.0 ** -19 + 2.0 ** -17
        base = acc[s].double().cpu().numpy()
        assert (got[lens[s]:] == 7.0).all() and (got0[lens[s]:] == 7.0).all()
        assert (np.abs(got0[:lens[s]] - w) <= rel * w + 1e-9).all()
        assert (np.abs(got[:lens[s]] - (w + 0.75 * base[:lens[s]])) <= rel * w + 2.0 ** -22 * (base[:lens[s]] + w) + 1e-9).all()
        # a row's weights add up to one
        rows = np.isfinite(l64[c.rows(s)]).sum()
        assert abs(w.sum() - rows) <= 1e-3 * max(rows, 1)


def test_weights_of_long_sequences_repeat_bit_by_bit():
    c = _case([1, 20], [9001, 3000], 8, 1, 128, 64, I8, BF, seed=12)
    _, lse = c.forward()
    a, b = (torch.zeros((2, 9001), device="cuda") for _ in range(2))
    for o in (a, b):
        c.att.moe_attn_weights(c.cells, c.q, lse, c.d_cu, c.d_lens, c.d_table, None, o, max_q=20, max_kv=9001)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    l64 = lse.double().cpu().numpy()
    for s, n in enumerate([9001, 3000]):
        w = oa.weights(c.q64[c.rows(s)], c.k64[s], l64[c.rows(s)], 0, c.scale)
        assert np.abs(a[s, :n].double().cpu().numpy() - w).max() <= 1e-4 * w.max()


# --- eviction ----------------------------------------------------------------------------
@pytest.mark.parametrize("lens,budget,recent", [
    ([1], 1, 0), ([5, 0, 9], 4, 2), ([300, 299, 301, 100], 100, 100), ([300, 50], 299, 0), ([4097, 1000, 5000], 777, 64),
    ([70000], 9001, 100), ([20, 30], 40, 3), ([512, 513], 512, 511),
])
@pytest.mark.parametrize("kind", ["ties", "spread", "odd"])
def test_evict(lens, budget, recent, kind):
    page, d, hkv = 16, 64, 1
    c = _case([0] * len(lens), lens, 1, hkv, d, page, I8 if kind == "ties" else BF, BF, seed=budget)
    g = np.random.default_rng(budget)
    width = max(lens) + 3
    acc = {"ties": g.integers(0, 4, (len(lens), width)) * 0.5,
           "spread": np.exp(g.normal(0, 8, (len(lens), width))),
           "odd": g.choice([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-42, 1.0, -2.0, 3e38], (len(lens), width))}[kind]
    acc = acc.astype(np.float32)
    per = -(-budget // page)
    extra = torch.full((len(lens) * per, page, c.cb), 0xEE, dtype=torch.uint8, device="cuda")
    cells = torch.cat([c.cells, extra])
    new_table = (torch.randperm(len(lens) * per).reshape(len(lens), per) + c.n_pages).to(torch.int32).cuda()
    keep = torch.full((len(lens), budget), 99, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    acc_out = torch.full((len(lens), budget), 7.0, device="cuda")
    old = cells.clone()
    c.att.moe_attn_evict(cells, torch.from_numpy(acc).cuda(), c.d_lens, c.d_table, recent, new_table, keep, new_lens, acc_out)
    c.att.moe_attn_sync()
    assert torch.equal(cells[:c.n_pages], old[:c.n_pages])
    cn, nt = cells.cpu().numpy(), new_table.cpu().numpy()
    for s, n in enumerate(lens):
        want = oa.evict(acc[s, :n], budget, recent)
        m = len(want)
        assert int(new_lens[s]) == m
        assert np.array_equal(keep[s].cpu().numpy(), np.concatenate([want, np.full(budget - m, -1)]))
        assert np.array_equal(acc_out[s].cpu().numpy(), np.concatenate([acc[s][want], np.zeros(budget - m, np.float32)]),
                              equal_nan=True)
        i = np.arange(m)
        assert np.array_equal(cn[nt[s][i // page], i % page], cn[c.table[s][want // page], want % page])
        left = np.arange(m, per * page)                   # cells beyond the kept ones are not written
        assert (cn[nt[s][left // page], left % page] == 0xEE).all()


def test_evict_reports_a_page_out_of_range():
    from expert_cached_decode_gb300 import MoeError
    c = _case([0], [100], 1, 1, 64, 16, BF, BF)
    acc = torch.rand(1, 100, device="cuda")
    keep = torch.zeros((1, 16), dtype=torch.int32, device="cuda")
    nl, ao = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((1, 16), device="cuda")
    before = c.cells.clone()
    c.att.moe_attn_evict(c.cells, acc, c.d_lens, c.d_table, 2, torch.tensor([[c.n_pages]], dtype=torch.int32, device="cuda"),
                         keep, nl, ao)
    with pytest.raises(MoeError, match="page id"):
        c.att.moe_attn_sync()
    assert torch.equal(c.cells, before) and int(nl[0]) == 16


# --- refusals of the binding ------------------------------------------------------------
def test_wrong_tensors_are_refused():
    c = _case([2], [40], 4, 2, 64, 16, BF, BF)
    out = torch.empty((2, 4, 64), dtype=BF, device="cuda")
    ok = (c.cells, c.q, c.d_cu, c.d_lens, c.d_table, out)

    def bad(i, t, match):
        a = list(ok)
        a[i] = t
        with pytest.raises(ValueError, match=match):
            c.att.moe_attn_forward(*a)

    bad(0, c.cells[:, :8], "cells")
    bad(0, c.cells.view(torch.int8), "uint8")
    bad(1, c.q.half(), "q must be")
    bad(1, c.q.transpose(1, 2), "shape")
    bad(1, torch.empty((2, 64, 4), dtype=BF, device="cuda").transpose(1, 2), "contiguous")
    bad(1, c.q.cpu(), "device tensor")
    bad(2, c.d_cu.long(), "cu_q")
    bad(2, c.d_cu[:1], "cu_q")
    bad(3, c.d_lens.cpu(), "kv_lens")
    bad(4, c.d_table.t(), "table")
    bad(5, out[:1], "out")
    with pytest.raises(ValueError, match="lse"):
        c.att.moe_attn_forward(*ok, lse=torch.empty((2, 4), dtype=BF, device="cuda"))
    from expert_cached_decode_gb300 import MoeError
    wide = torch.empty((2, 5, 68), dtype=BF, device="cuda").flatten(1)[:, 4:4 + 256].unflatten(1, (4, 64))
    with pytest.raises(MoeError, match="16-byte"):
        c.att.moe_attn_forward(c.cells, wide, c.d_cu, c.d_lens, c.d_table, out)
    with pytest.raises(MoeError, match="acc_stride"):
        c.att.moe_attn_weights(c.cells, c.q, torch.zeros((2, 4), device="cuda"), c.d_cu, c.d_lens, c.d_table, None,
                               torch.zeros((1, 20), device="cuda"), max_kv=48)


# --- shapes that meet each kernel's edges ---------------------------------------------------
@pytest.mark.parametrize("hq,hkv", [(5, 1), (14, 2), (32, 1), (3, 3)])
@pytest.mark.parametrize("n", [1, 2, 6, 7, 26, 60])
@pytest.mark.parametrize("kv", [BF, I8])
def test_group_sizes_against_row_tiles(hq, hkv, n, kv):
    # rows per K/V head from 1 to 1,920: single row tiles, two tiles of 16, one of 128, several of 256, ragged ends
    c = _case([n, 1], [n + 300, 140], hq, hkv, 64, 16, kv, BF, seed=hq * n)
    out, lse = _check(c, max_q=n)
    acc = torch.full((2, n + 300), 7.0, device="cuda")
    c.att.moe_attn_weights(c.cells, c.q, lse, c.d_cu, c.d_lens, c.d_table, None, acc, max_q=n)
    c.att.moe_attn_sync()
    for s in range(2):
        w = oa.weights(c.q64[c.rows(s)], c.k64[s], lse[c.rows(s)].double().cpu().numpy(), 0, c.scale)
        got = acc[s, :c.kv_lens[s]].double().cpu().numpy()
        assert np.abs(got - w).max() <= 1e-4 * w.max()


@pytest.mark.parametrize("page", [1, 24, 100, 64])
@pytest.mark.parametrize("kv,io,d", [(BF, BF, 128), (I8, BF, 128), (FP, FP, 64), (I8, FP, 64)])
def test_chunks_over_pages_with_and_without_boxes(page, kv, io, d):
    _check(_case([150, 40], [700, 431], 4, 1, d, page, kv, io, seed=page + d))


@pytest.mark.parametrize("kv,d", [(BF, 128), (I8, 128), (BF, 64), (I8, 64)])
def test_items_cut_at_every_place(kv, d):
    # sequences of 1 to 20 tiles with 40 rows (two streams on alternate tiles), then with 200 (two streams on two halves)
    lens = [128 * k + (k * 37) % 128 + 60 for k in range(1, 20)]
    _check(_case([10] * 19, lens, 8, 2, d, 32, kv, BF, seed=d), max_q=10)
    _check(_case([50] * 8, lens[:8], 8, 2, d, 32, kv, BF, seed=d), max_q=50)


def test_calls_of_every_kind_on_one_handle():
    # the work space is shared: what one call leaves in it reaches no other
    kinds = [([1] * 5, 1), ([4] * 5, 4), ([10] * 5, 10), ([70, 1, 9, 2, 1], 70), ([40] * 5, 40)]
    cases = [_case(n, [900, 333, 2000, 64, 801], 8, 2, 128, 32, I8, BF, seed=i) for i, (n, _) in enumerate(kinds)]
    att = cases[0].att
    want = []
    for c, (_, mq) in zip(cases, kinds):
        want.append(c.forward(max_q=mq))
        c.att.moe_attn_sync()
    for i in list(range(5)) * 2 + [4, 3, 2, 1, 0]:
        cases[i].att = att
        out, lse = cases[i].forward(max_q=kinds[i][1])
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_queries_of_another_sequence_do_not_matter():
    # the tiles that hold a sequence's last rows hold its neighbour's first ones too
    c = _case([50, 50], [300, 200], 8, 2, 128, 32, BF, BF, seed=1)
    out, lse = c.forward()
    acc = torch.zeros((2, 300), device="cuda")
    c.att.moe_attn_weights(c.cells, c.q, lse, c.d_cu, c.d_lens, c.d_table, None, acc)
    c.q = c.q.clone()
    c.q[50:] = float("nan")
    lse2 = lse.clone()
    lse2[50:] = float("nan")
    acc2 = torch.zeros((2, 300), device="cuda")
    c.att.moe_attn_weights(c.cells, c.q, lse2, c.d_cu, c.d_lens, c.d_table, None, acc2)
    out2, _ = c.forward()
    torch.cuda.synchronize()
    assert torch.equal(acc[0], acc2[0]) and torch.equal(out[:50], out2[:50])


def test_a_strided_cache_with_wide_cells_and_tiny_and_huge_scales():
    c = _case([1, 30], [200, 200], 8, 1, 128, 16, I8, BF, seed=3, pad=32)
    # V scales from 2^-30 to 2^30: the output's own scale, no overflow and no loss
    for e in (-30, 30):
        cells = c.cells.clone().view(torch.uint8)
        f = cells.reshape(-1, c.cb)[:, 256:264].contiguous().view(torch.float32)
        f[:, 1] *= 2.0 ** e
        cells.reshape(-1, c.cb)[:, 256:264] = f.view(torch.uint8)
        a, _ = c.forward(max_q=30)
        c.cells, keep = cells, c.cells
        b, _ = c.forward(max_q=30)
        c.cells = keep
        x, y = a.double(), b.double() / 2.0 ** e
        assert torch.isfinite(y).all()
        assert ((x - y).abs() <= 2.0 ** -7 * x.abs().max(-1, keepdim=True).values).all()


@pytest.mark.parametrize("n,recent", [(800_001, 100), (1_000_000, 0)])
def test_evict_from_more_cells_than_keys_fit_on_chip(n, recent):
    c = _case([0], [64], 1, 1, 64, 64, BF, BF)          # one page of cells, which every entry of the long table names
    pages = -(-n // 64)
    cells = torch.cat([c.cells, torch.zeros((20, 64, c.cb), dtype=torch.uint8, device="cuda")])
    table = torch.full((1, pages), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    acc = np.exp(np.random.default_rng(n).normal(0, 3, (1, n))).astype(np.float32)
    acc[0, ::7] = acc[0, 0]                              # ties
    budget = 1200
    keep = torch.zeros((1, budget), dtype=torch.int32, device="cuda")
    new_lens, acc_out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((1, budget), device="cuda")
    new_table = torch.arange(c.n_pages, c.n_pages + 19, dtype=torch.int32, device="cuda")[None]
    c.att.moe_attn_evict(cells, torch.from_numpy(acc).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), table,
                         recent, new_table, keep, new_lens, acc_out)
    c.att.moe_attn_sync()
    want = oa.evict(acc[0], budget, recent)
    assert np.array_equal(keep[0].cpu().numpy(), want) and int(new_lens[0]) == budget
    assert np.array_equal(acc_out[0].cpu().numpy(), acc[0][want])
    got = cells[c.n_pages:].reshape(-1, c.cb)[:budget]
    assert torch.equal(got, c.cells[int(c.table[0, 0])][torch.from_numpy(want % 64).cuda()])


@pytest.mark.parametrize("kv,io,d", [(BF, BF, 128), (I8, BF, 128), (FP, FP, 64), (I8, FP, 64)])
@pytest.mark.parametrize("n", [20, 70])
def test_references_that_grow_within_a_tile(kv, io, d, n):
    # scores of a spread of some 30 bits: a row's largest so far is outgrown by far more than the slack, again and again,
    # also between the halves of one tile, where the first half's probabilities have been written already
    _check(_case([n, n], [900, 130], 8, 2, d, 32, kv, io, seed=d + n, std=5.0 if d == 128 else 6.0))


@pytest.mark.parametrize("kv,d,n,hq", [(BF, 128, 5, 8), (I8, 128, 6, 8), (I8, 64, 16, 3), (BF, 64, 9, 4), (FP, 128, 7, 5)])
def test_weights_of_three_row_tiles_over_many_cells(kv, d, n, hq):
    # 33 to 48 rows, and cells enough for every warp of the few-row kernel
    io = FP if kv == FP else BF
    c = _case([n, 1], [81_000, 45], hq, 1, d, 64, kv, io, seed=n)
    _, lse = c.forward(max_q=n)
    acc = torch.full((2, 81_000), 3.0, device="cuda")
    c.att.moe_attn_weights(c.cells, c.q, lse, c.d_cu, c.d_lens, c.d_table, acc, acc, decay=0.5, max_q=n)
    c.att.moe_attn_sync()
    for s, length in enumerate([81_000, 45]):
        w = oa.weights(c.q64[c.rows(s)], c.k64[s], lse[c.rows(s)].double().cpu().numpy(), 0, c.scale) + 1.5
        assert np.abs(acc[s, :length].double().cpu().numpy() - w).max() <= 1e-4 * w.max()
    assert (acc[1, 45:] == 3.0).all()


@pytest.mark.parametrize("seqs", [9, 17, 40])
def test_evictions_of_many_long_sequences(seqs):
    # as many sequences as make the clusters 8, 4 and 2 wide
    n, budget = 9000, 300
    c = _case([0], [64], 1, 1, 64, 64, BF, BF)
    pages = -(-n // 64)
    cells = torch.cat([c.cells, torch.zeros((seqs * 5, 64, c.cb), dtype=torch.uint8, device="cuda")])
    table = torch.full((seqs, pages), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    g = np.random.default_rng(seqs)
    acc = np.exp(g.normal(0, 2, (seqs, n))).astype(np.float32).round(2)
    lens = [n - 100 * i for i in range(seqs)]
    keep = torch.zeros((seqs, budget), dtype=torch.int32, device="cuda")
    new_lens, acc_out = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros((seqs, budget), device="cuda")
    new_table = torch.arange(c.n_pages, c.n_pages + seqs * 5, dtype=torch.int32, device="cuda").reshape(seqs, 5)
    c.att.moe_attn_evict(cells, torch.from_numpy(acc).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), table, 20,
                         new_table, keep, new_lens, acc_out)
    c.att.moe_attn_sync()
    for s in range(seqs):
        want = oa.evict(acc[s, :lens[s]], budget, 20)
        assert np.array_equal(keep[s].cpu().numpy(), want) and np.array_equal(acc_out[s].cpu().numpy(), acc[s][want])
