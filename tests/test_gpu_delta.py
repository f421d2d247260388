"""The gated delta rule on the GPU against the 64-bit oracle: lengths from none
to several chunks, head layouts, types, strides, slots, refusals."""

import numpy as np
import pytest
import torch

from delta_helpers import Case, unit
from expert_cached_decode_gb300 import GatedDelta, MoeError
from oracle import delta as od

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("lens", [[1], [2], [8], [9], [1, 1, 1], [5, 5], [0, 1, 0, 7], [17, 3]])
@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 64, HF), (128, 64, HF), (64, 128, BF)])
def test_steps(lens, dk, dv, dtype):
    c = Case(lens, dk=dk, dv=dv, dtype=dtype, pad=3, seed=len(lens))
    c.check(c.forward(max_q=max(lens)))


@pytest.mark.parametrize("lens", [[63], [64], [65], [128, 1], [130, 64, 0, 40], [1, 200, 1, 33], [321]])
@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (128, 128, HF), (64, 64, HF), (128, 64, BF), (64, 128, BF)])
def test_chunks(lens, dk, dv, dtype):
    c = Case(lens, dk=dk, dv=dv, dtype=dtype, pad=2, seed=sum(lens))
    c.check(c.forward(max_q=max(lens)))
    c.check(c.forward())                       # the bound left open: another kernel may take it, the result holds


@pytest.mark.parametrize("lens", [[960], [1031], [2000, 1, 0, 1300], [64 * 15, 64 * 15 + 1], [3300]])
@pytest.mark.parametrize("dk,dv,dtype,hk,hv", [(128, 128, BF, 1, 1), (64, 64, HF, 1, 2), (128, 64, BF, 2, 2), (64, 128, BF, 1, 3)])
def test_parts(lens, dk, dv, dtype, hk, hv):
    # few heads: long sequences are cut into parts that go through side by side
    c = Case(lens, hk=hk, hv=hv, dk=dk, dv=dv, dtype=dtype, pad=1, seed=len(lens), decay=0.01, keep=(0,))
    c.check(c.forward(max_q=max(lens)))
    c.g64[:] = 0.0                             # nothing is forgotten: every part matters to the end
    c.check(c.forward())


@pytest.mark.parametrize("lens,hk,hv", [([5000, 70, 3000], 64, 128), ([9000], 64, 64), ([40] * 100, 64, 128)])
def test_more_chunks_than_the_work_space_holds(lens, hk, hv):
    # the state goes on from one window of chunks to the next; against the same call token by token
    c = Case(lens, hk=hk, hv=hv, dk=64, dv=64, seed=3, decay=0.003, pad=1)
    a, b = c.forward(max_q=1), c.forward()
    torch.cuda.synchronize()
    # far above what rounding makes of either (2^-17 of what goes into a column), far below a chunk that is missing
    for s in range(c.S):
        x, y = a["state"][c.s_out[s]].double(), b["state"][c.s_out[s]].double()
        assert ((x - y).norm(dim=1) <= 2.0 ** -13 * x.norm(dim=1) + 1e-6).all()
    x, y = a["out"].double(), b["out"].double()
    assert ((x - y).norm(dim=2) <= 2.0 ** -6 * x.norm(dim=2) + 1e-6).all()
    c.op.moe_delta_sync()


@pytest.mark.parametrize("hk,hv", [(1, 1), (3, 3), (1, 5), (5, 10), (16, 32)])
@pytest.mark.parametrize("n", [1, 70])
def test_heads(hk, hv, n):
    c = Case([n, 2], hk=hk, hv=hv, seed=hv)
    c.check(c.forward(max_q=n))


@pytest.mark.parametrize("n", [4, 90])
def test_slots(n):
    # from zeros, to nowhere, to another slot; sequences without tokens carry their state over, or zeros
    c = Case([n, n, n + 1, 0, 0, 0, 1], fresh=(0, 4), drop=(1, 5), keep=(2, 3), seed=5)
    c.check(c.forward())
    c.op.moe_delta_sync()


@pytest.mark.parametrize("n", [3, 100])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_not_normalized(n, dtype):
    c = Case([n, 2 * n], normalize=False, dtype=dtype, scale=0.25, seed=2)
    c.check(c.forward())


@pytest.mark.parametrize("n", [7, 150])
def test_decays_from_none_to_all(n):
    c = Case([n], seed=3)
    c.g64[:] = 0.0
    c.check(c.forward())
    c.g64[:] = -30.0                           # every token forgets nearly all
    c.check(c.forward())
    c.g64[:] = 0.0
    c.g64[n // 2] = -np.inf                    # one token forgets all
    c.g64[n // 3, 1] = -200.0
    c.check(c.forward())


@pytest.mark.parametrize("n", [9, 192])
def test_the_same_key_again_and_again(n):
    # (1 + A)^-1 of keys that are all alike: powers of A would cancel
    c = Case([n], seed=4, same_keys=True)
    c.g64[:] = 0.0
    c.b64[:] = 1.0
    c.check(c.forward())
    c.b64[:] = 0.0                             # nothing is written at all
    c.check(c.forward())


@pytest.mark.parametrize("n", [3, 80])
def test_large_and_small_values(n):
    c = Case([n, n], seed=6, fresh=(1,))
    c.st64[c.s_in[0]] *= 2.0 ** 40
    c.st64[c.s_in[0]][:, :, ::2] *= 2.0 ** -60           # columns of very different sizes
    c.check(c.forward())
    c = Case([n], seed=7)
    c.x[:, c.nq:2 * c.nq] *= 2.0 ** -40                  # keys far below eps: next to nothing is written
    c.x64 = c.x.double().cpu().numpy()
    c.check(c.forward())
    c = Case([n], seed=7)
    c.x[:, c.nq:2 * c.nq] *= 2.0 ** 40
    c.x[:, 2 * c.nq:] *= 2.0 ** 30
    c.x64 = c.x.double().cpu().numpy()
    c.check(c.forward())


def test_rows_are_apart():
    # a NaN in one value column, in one head's state and in padding reaches nothing else
    for n in (5, 130):
        c = Case([n, n], pad=4, seed=8)
        want = c.forward()
        bad = c.device()
        x = c.x.clone()
        x[c.T:] = float("nan")
        x[2, 2 * c.nq + 3] = float("nan")                # head 0, column 3, from token 2 of sequence 0
        bad["state"][c.s_in[1], 2] = float("nan")        # head 2 of sequence 1
        q, k, v = c.views(x)
        c.op.moe_delta_forward(q, k, v, **bad)
        a, b = want["out"].clone(), bad["out"].clone()
        for z in (a, b):
            z[:n, 0, 3] = 0                              # (within its chunk it may reach the tokens before)
            z[n:2 * n, 2] = 0
        assert torch.equal(a, b)
        assert torch.isnan(bad["out"][2:n, 0, 3]).all() and torch.isnan(bad["out"][n:2 * n, 2]).all()
        a, b = want["state"].clone(), bad["state"].clone()
        for z in (a, b):
            z[c.s_out[0], 0, :, 3] = 0
            z[c.s_out[1], 2] = 0
        assert torch.equal(a, b)


def test_a_prompt_in_parts_is_the_prompt():
    # the state carries over: 200 tokens at once, and as 70 + 1 + 1 + 128
    c = Case([200], seed=9)
    whole = c.forward()
    c.check(whole)
    d = c.device()
    q, k, v = c.views(c.x)
    at = 0
    for n in (70, 1, 1, 128):
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        c.op.moe_delta_forward(q[at:at + n], k[at:at + n], v[at:at + n], d["g"][at:at + n], d["beta"][at:at + n], d["state"],
                               d["out"][at:at + n], cu, d["slots_in"], d["slots_out"], max_q=n)
        at += n
    c.check(d)


def test_repeats_bitwise_and_on_any_stream():
    c = Case([150, 1, 7, 64], seed=10)
    want = c.forward()
    s = torch.cuda.Stream()
    for _ in range(3):
        d = c.device()
        torch.cuda.synchronize()
        c.forward(d, stream=s)
        s.synchronize()
        assert torch.equal(d["out"], want["out"]) and torch.equal(d["state"], want["state"])


def test_captured_and_replayed_after_the_batch_changed():
    c = Case([100, 3, 0, 1], pad=60, seed=11)
    d = c.device()
    c.forward(c.device())                     # (first use of the kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(d)
    for lens, seed in (([100, 3, 0, 1], 11), ([1, 1, 1, 1], 12), ([10, 70, 80, 4], 13)):
        n = Case(lens, pad=164 - sum(lens), seed=seed)
        f = n.device()
        for name in d:
            d[name].copy_(f[name])
        c.x.copy_(n.x)
        graph.replay()
        n.check(d)


def test_bad_slots_and_offsets_are_left_out_and_reported():
    for n in (2, 100):
        c = Case([n, n, n, n], seed=12)
        d = c.device()
        d["slots_in"][1] = c.n_slots           # counts as -1
        d["slots_out"][2] = -2
        c.forward(d)
        with pytest.raises(MoeError, match="slot out of range"):
            c.op.moe_delta_sync()
        c.op.moe_delta_sync()                  # once
        c.s_in[1], c.s_out[2] = -1, -1
        c.check(d)
        c = Case([n, n], pad=5, seed=13)
        d = c.device()
        d["cu"][2] = 10 ** 6                   # cut to the rows that there are
        c.forward(d)
        with pytest.raises(MoeError, match="offset"):
            c.op.moe_delta_sync()
        torch.cuda.synchronize()


def test_slots_that_clash_are_not_written():
    for n in (2, 100):
        c = Case([n, n, n, 0, 0], seed=14)
        d = c.device()
        c.s_out[1] = c.s_out[0]                # an earlier one writes it
        c.s_out[2] = c.s_in[1]                 # another one reads it
        c.s_in[4] = c.s_out[4] = c.s_in[3]     # padding that shares a slot: not a clash
        d["slots_in"].copy_(torch.from_numpy(c.s_in))
        d["slots_out"].copy_(torch.from_numpy(c.s_out))
        c.forward(d)
        with pytest.raises(MoeError, match="another"):
            c.op.moe_delta_sync()
        c.check(d, writes=(0, 3, 4))


def test_nothing_to_do():
    c = Case([], pad=4)
    c.check(c.forward())
    c = Case([0, 0], pad=0)
    c.check(c.forward())


def test_refusals():
    c = Case([4, 2], seed=15)
    q, k, v = c.views(c.x)
    ok = c.device()
    bad = lambda exc, words, q=q, k=k, v=v, **kw: _refused(c, exc, words, q, k, v, {**ok, **kw})
    bad(ValueError, "q must be", q=q.float())
    bad(ValueError, "shape", k=k[:3])
    bad(ValueError, "contiguous", v=v.transpose(0, 1).contiguous().transpose(0, 1))
    bad(ValueError, "g must", g=ok["g"].double())
    bad(ValueError, "state must", state=ok["state"][:, :, :, :64])
    bad(ValueError, "out must", out=ok["out"][:5])
    bad(ValueError, "cu must", cu=ok["cu"].long())
    bad(ValueError, "slots_out must", slots_out=ok["slots_out"][:1])
    bad(ValueError, "beta must", beta=ok["beta"].cpu())
    wide = torch.zeros(6, 4 * 128 + 4, dtype=BF, device="cuda")
    bad(MoeError, "16-byte", q=wide[:, 4:260].view(6, 2, 128))
    over = torch.zeros(6, 4, 128, dtype=BF, device="cuda")
    bad(MoeError, "overlaps", v=over, out=over)
    n = 4097
    z = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    bad(MoeError, "n_seqs", cu=z, slots_in=z[:n], slots_out=z[:n])
    c.op.moe_delta_sync()


def _refused(c, exc, words, q, k, v, kw):
    before = kw["state"].clone()
    with pytest.raises(exc, match=words):
        c.op.moe_delta_forward(q, k, v, **kw)
    torch.cuda.synchronize()
    assert torch.equal(kw["state"], before)


# ------------------------------------------------------- convolution, gates --
def _prep(lens, hk=1, hv=3, dk=64, dv=64, taps=4, dtype=BF, seed=0, pad=0, fresh=(), keep=(), bias=True, gap=8):
    g = np.random.default_rng(seed)
    S, T = len(lens), int(sum(lens))
    op = GatedDelta(hk, hv, dk, dv, dtype=dtype, taps=taps)
    C = op.channels
    t = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).to(dtype).cuda()
    order = g.permutation(2 * S + 1).astype(np.int32)
    s_in, s_out = order[:S].copy(), order[:S].copy()
    for s in keep:
        s_out[s] = order[S + s]
    for s in fresh:
        s_in[s] = -1
    ab = t(T + pad, 2 * hv)
    d = dict(x=t(T + pad, C + gap)[:, :C], conv_w=t(C, taps), conv_bias=t(C) if bias else None, conv_state=t(2 * S + 1, taps - 1, C),
             y=torch.full((T + pad, C), 7.0, dtype=dtype, device="cuda"), a=ab[:, :hv], b=ab[:, hv:],
             a_log=torch.from_numpy(g.standard_normal(hv).astype(np.float32)).cuda(),
             dt_bias=torch.from_numpy(g.standard_normal(hv).astype(np.float32)).cuda(),
             g=torch.full((T + pad, hv), 7.0, device="cuda"), beta=torch.full((T + pad, hv), 7.0, device="cuda"),
             cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda(),
             slots_in=torch.from_numpy(s_in).cuda(), slots_out=torch.from_numpy(s_out).cuda())
    return op, d, lens, s_in, s_out


def _check_prep(op, d, lens, s_in, s_out, before):
    torch.cuda.synchronize()
    f = lambda t: t.double().cpu().numpy()
    x, w, b = f(d["x"]), f(d["conv_w"]), None if d["conv_bias"] is None else f(d["conv_bias"])
    y, st, old = f(d["y"]), f(d["conv_state"]), f(before)
    want = old.copy()
    at = 0
    for s, n in enumerate(lens):
        o = old[s_in[s]] if s_in[s] >= 0 else np.zeros_like(old[0])
        r, new, mag = od.conv(x[at:at + n], w, b, o)
        # one rounding; before it fp32 sums of at most five terms (2^-21 of their magnitudes; silu's slope is below 1.1)
        assert (np.abs(y[at:at + n] - r) <= unit(op.dtype) * 1.01 * np.abs(r) + 2.0 ** -20 * mag + 2.0 ** -24).all()
        if s_out[s] >= 0:
            want[s_out[s]] = new
        at += n
    assert np.array_equal(st, want)
    g, beta = od.gates(f(d["a"]), f(d["b"]), f(d["a_log"]), f(d["dt_bias"]))
    assert np.allclose(f(d["g"])[:at], g[:at], rtol=2.0 ** -20, atol=2.0 ** -40)
    assert np.allclose(f(d["beta"])[:at], beta[:at], rtol=2.0 ** -20, atol=0)
    for z in (d["y"], d["g"], d["beta"]):
        assert (z[at:] == 7.0).all()


@pytest.mark.parametrize("lens", [[1], [2], [3, 1, 0, 2], [0, 0, 5], [40, 1, 1, 19, 2], [1] * 40, [700]])
@pytest.mark.parametrize("taps,dtype", [(4, BF), (3, HF), (2, BF)])
def test_prepare(lens, taps, dtype):
    op, d, *rest = _prep(lens, taps=taps, dtype=dtype, seed=len(lens), pad=3, bias=taps != 3)
    before = d["conv_state"].clone()
    op.moe_delta_prepare(**d)
    _check_prep(op, d, *rest, before)
    op.moe_delta_sync()


def test_prepare_long_runs():
    # enough tokens that a thread takes a run of them; sequences begin and end at every place of a run
    lens = [1, 2, 3, 15, 16, 17, 0, 33, 5] * 60 + [9000]
    op, d, *rest = _prep(lens, hk=4, hv=4, dk=128, dv=128, seed=3, fresh=(0, 7, 20), keep=(3, 6, 30))
    before = d["conv_state"].clone()
    op.moe_delta_prepare(**d)
    _check_prep(op, d, *rest, before)


def test_prepare_slots():
    op, d, lens, s_in, s_out = _prep([2, 5, 0, 0, 1, 3], fresh=(0, 3), keep=(1, 2, 3), seed=4)
    s_out[4] = s_in[5]                         # sequence 5 reads it: not written, by neither
    d["slots_out"].copy_(torch.from_numpy(s_out))
    d["slots_in"][1] = 10 ** 6
    before = d["conv_state"].clone()
    op.moe_delta_prepare(**d)
    with pytest.raises(MoeError, match="another"):
        op.moe_delta_sync()
    s_out[4] = s_out[5] = s_in[1] = -1         # (and 4, the earlier one, would write the slot of 5)
    _check_prep(op, d, lens, s_in, s_out, before)


def test_prepare_parts_and_halves():
    # a prompt in parts gives the same rows; the convolution and the gates alone too
    op, d, *rest = _prep([50], seed=5)
    before = d["conv_state"].clone()
    op.moe_delta_prepare(**d)
    y, st = d["y"].clone(), d["conv_state"].clone()
    d["conv_state"].copy_(before)
    d["y"].fill_(0)
    at = 0
    for n in (1, 2, 30, 1, 16):
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        op.moe_delta_prepare(d["x"][at:at + n], d["conv_w"], d["conv_bias"], d["conv_state"], d["y"][at:at + n], None, None, None,
                             None, None, None, cu, d["slots_in"], d["slots_out"])
        at += n
    assert torch.equal(d["y"], y) and torch.equal(d["conv_state"], st)
    g = d["g"].clone()
    d["g"].zero_()
    op.moe_delta_prepare(None, None, None, None, None, *(d[k] for k in ("a", "b", "a_log", "dt_bias", "g", "beta", "cu", "slots_in", "slots_out")))
    assert torch.equal(d["g"], g)
    op.moe_delta_sync()


def test_prepare_nothing():
    op, d, *rest = _prep([0, 0, 0], fresh=(1,), keep=(0, 1), seed=8)
    before = d["conv_state"].clone()
    op.moe_delta_prepare(**d)
    _check_prep(op, d, *rest, before)
    op, d, *rest = _prep([], seed=8, pad=2)
    before = d["conv_state"].clone()
    op.moe_delta_prepare(**d)
    _check_prep(op, d, *rest, before)


def test_gates_at_their_ends():
    op, d, *rest = _prep([6], seed=6)
    d["a"][:, 0] = torch.tensor([100.0, -100.0, 0.0, 1e4, -1e4, float("nan")], dtype=BF)
    d["b"][:, 0] = torch.tensor([100.0, -100.0, 0.0, 1e4, -1e4, float("nan")], dtype=BF)
    op.moe_delta_prepare(**d)
    g, beta = d["g"][:, 0].double().cpu().numpy(), d["beta"][:, 0].double().cpu().numpy()
    with np.errstate(over="ignore"):
        wg, wb = od.gates(d["a"][:, 0].double().cpu().numpy(), d["b"][:, 0].double().cpu().numpy(), d["a_log"][0].item(),
                          d["dt_bias"][0].item())
    assert np.allclose(g, wg, rtol=2.0 ** -20, atol=2.0 ** -100, equal_nan=True)
    assert np.allclose(beta, wb, rtol=2.0 ** -20, atol=2.0 ** -100, equal_nan=True)


def test_prepare_refusals():
    op, d, *rest = _prep([4], seed=7)
    for words, kw in [("x must", dict(x=d["x"].float())), ("conv_w must", dict(conv_w=d["conv_w"][:, :3])),
                      ("conv_state must", dict(conv_state=d["conv_state"][:, :2])), ("y must", dict(y=d["y"][:3])),
                      ("strides", dict(a=d["a"].contiguous())), ("a_log must", dict(a_log=d["a_log"].double())),
                      ("x or a", dict(x=None, a=None))]:
        with pytest.raises(ValueError, match=words):
            op.moe_delta_prepare(**{**d, **kw})
    y = torch.zeros(4, op.channels, dtype=BF, device="cuda")
    with pytest.raises(MoeError, match="overlaps"):
        op.moe_delta_prepare(**{**d, "x": y, "y": y})
    none = GatedDelta(1, 3, 64, 64, taps=0)
    with pytest.raises(MoeError, match="no convolution"):
        none.taps = 4
        none.moe_delta_prepare(**d)
