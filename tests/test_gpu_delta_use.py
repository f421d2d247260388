"""The gated delta rule as programs use it: tensors side by side in one
allocation, threads, streams, graphs on one handle, and a layer's calls in a row."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from delta_helpers import Case
from expert_cached_decode_gb300 import MoeError, moe_norm_block, moe_norm_gated
from oracle import delta as od

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 4, 128, 128), (2, 2, 128, 64), (1, 1, 64, 128)])
def test_out_directly_behind_or_before_the_inputs(n, hk, hv, dk, dv):
    # rows of q, k, v and out that touch, in either order, are apart: none may count with another's width
    c = Case([n], hk=hk, hv=hv, dk=dk, dv=dv, seed=n)
    q, k, v = (t.contiguous() for t in c.views(c.x))
    for order in ("qkvo", "ovkq", "vokq", "kqov", "vqok"):
        d = c.device()
        t = dict(q=q, k=k, v=v, o=d["out"])
        flat = torch.empty(sum(x.numel() for x in t.values()), dtype=c.dtype, device="cuda")
        at, got = 0, {}
        for name in order:
            got[name] = flat[at:at + t[name].numel()].view(t[name].shape)
            got[name].copy_(t[name])
            at += t[name].numel()
        d["out"] = got["o"]
        c.op.moe_delta_forward(got["q"], got["k"], got["v"], **d)
        c.check(d)


@pytest.mark.parametrize("n", [3, 70])
def test_rows_and_slots_far_apart(n):
    # offsets past 2^31 elements: token strides of 2^25 (70 tokens) or 2^30 (3), and the last slots of a state of 9 GB
    hk, hv = 2, 4
    c = Case([n], hk=hk, hv=hv, seed=n, dk=128, dv=128)
    stride = 2 ** 30 if n == 3 else 2 ** 25
    flat = torch.zeros((n - 1) * stride + c.x.shape[1], dtype=c.dtype, device="cuda")
    x = flat.as_strided(c.x.shape, (stride, 1))
    x.copy_(c.x)
    q, k, v = c.views(x)
    assert (n - 1) * stride >= 2 ** 31
    d = c.device()
    slots = 2 ** 31 // (hv * 128 * 128) + 2
    big = torch.zeros((slots, hv, 128, 128), device="cuda")
    big[slots - 1].copy_(d["state"][c.s_in[0]])
    small = d["state"]
    d["state"] = big
    d["slots_in"].fill_(slots - 1)
    d["slots_out"].fill_(slots - 2)
    c.op.moe_delta_forward(q, k, v, **d)
    c.op.moe_delta_sync()
    assert torch.equal(big[slots - 1], small[c.s_in[0]]) and not big[:slots - 2].any()
    small[c.s_out[0]].copy_(big[slots - 2])
    c.check({**d, "state": small})


@pytest.mark.parametrize("n", [1535, 1536, 1537, 1920, 3000])
def test_where_sequences_begin_to_be_cut(n):
    c = Case([n, 5], hk=1, hv=2, seed=n, decay=0.02, pad=3, fresh=(1,))
    c.check(c.forward(max_q=n))


def test_a_cut_call_and_its_rows_one_after_another():
    # a sequence beside others that are not cut; the same call again gives the same bits
    c = Case([2500, 64, 0, 1, 24, 25, 1700], hk=1, hv=2, seed=5, decay=0.02)
    a, b = c.forward(), c.forward()
    torch.cuda.synchronize()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["state"], b["state"])
    c.check(a)


def test_threads_on_one_stream_get_their_own_results():
    kinds = [[1] * 5, [200, 3], [2000], [30, 90, 64]]
    cases = [Case(n, hk=2, hv=4, seed=i) for i, n in enumerate(kinds)]
    op = cases[0].op
    stream = torch.cuda.Stream()

    def call(c):
        d = c.device()
        q, k, v = c.views(c.x)
        torch.cuda.current_stream().synchronize()
        op.moe_delta_forward(q, k, v, **d, stream=stream)
        return d

    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            got = [call(cases[i]) for _ in range(25)]
            stream.synchronize()
            wrong.extend(i for g in got if not (torch.equal(g["out"], want[i]["out"]) and torch.equal(g["state"], want[i]["state"])))
        except Exception as e:                       # a thread's failure is the test's
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    op.moe_delta_sync()
    assert not errors and not wrong, (errors, wrong)


def test_two_graphs_on_one_handle():
    # replayed in turn on one stream, with eager calls between: each leaves its own results in spite of the shared work space
    cases = [Case([300, 2], hk=2, hv=4, seed=1), Case([40, 1800], hk=2, hv=4, seed=2)]
    op = cases[0].op
    want, held = [], []
    for c in cases:
        q, k, v = c.views(c.x)
        d = c.device()
        op.moe_delta_forward(q, k, v, **d)
        torch.cuda.synchronize()
        want.append((d["out"].clone(), d["state"].clone()))
        d, first = c.device(), c.device()["state"]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            op.moe_delta_forward(q, k, v, **d)
        held.append((g, d, first))
    for i in (0, 1, 1, 0, 0, 1):
        g, d, first = held[i]
        d["state"].copy_(first)
        d["out"].zero_()
        g.replay()
        other = cases[1 - i]
        e = other.device()
        op.moe_delta_forward(*other.views(other.x), **e)
        torch.cuda.synchronize()
        c = cases[i]
        assert torch.equal(d["out"][:c.T], want[i][0][:c.T]) and torch.equal(d["state"], want[i][1])
        assert torch.equal(e["out"], want[1 - i][0]) and torch.equal(e["state"], want[1 - i][1])


def test_two_handles_on_two_streams():
    cases = [Case([500, 64, 1], hk=2, hv=4, seed=3), Case([1700], hk=2, hv=4, seed=4)]
    want = [c.forward() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[c.device() for _ in range(8)] for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, s, g in zip(cases, streams, got):
            c.forward(g[i], stream=s)
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(g["out"], w["out"]) and torch.equal(g["state"], w["state"])


def test_norms_refuse_overlaps_and_take_neighbours():
    n, d = 4, 64
    w = torch.ones(d, dtype=BF, device="cuda")
    flat = torch.randn(5 * n * d, device="cuda").to(BF)
    y, h, gate, ho, x = (flat[i * n * d:(i + 1) * n * d].view(n, d) for i in range(5))
    moe_norm_block(y, h, ho, x, pre_w=w, gate=gate)                        # side by side: apart
    moe_norm_block(y, h, h, x, pre_w=w, gate=gate)                         # in place
    shifted = flat[2 * d:(n + 2) * d].view(n, d)                           # two rows into y, two into h
    before = flat.clone()
    for kw in (dict(h_out=y), dict(x=y), dict(x=h), dict(h_out=gate), dict(h_out=ho, x=ho), dict(h_out=shifted), dict(x=shifted),
               dict(pre_w=x[0]), dict(post_w=ho[1])):
        with pytest.raises(MoeError, match="overlaps"):
            moe_norm_block(**{**dict(y=y, h=h, h_out=ho, x=x, pre_w=w, gate=gate), **kw})
    o, z = y.view(n, 1, d), h.view(n, 1, d)
    for kw in (dict(out=z), dict(out=shifted.view(n, 1, d)), dict(w=ho[0])):
        with pytest.raises(MoeError, match="overlaps"):
            moe_norm_gated(**{**dict(o=o, z=z, w=w, out=ho.view(n, 1, d)), **kw})
    torch.cuda.synchronize()
    assert torch.equal(flat, before)


def test_norm_rows_far_apart():
    # row strides of 2^30 elements: offsets past 2^31
    n, d = 3, 256
    far = torch.zeros((n - 1) * 2 ** 30 + d, dtype=BF, device="cuda").as_strided((n, d), (2 ** 30, 1))
    near = torch.randn(n, d, device="cuda").to(BF)
    far.copy_(near)
    w = torch.ones(d, dtype=BF, device="cuda")
    a, b = [torch.empty(n, d, dtype=BF, device="cuda") for _ in range(2)], [torch.empty(n, d, dtype=BF, device="cuda") for _ in range(2)]
    moe_norm_block(near, near, *a, pre_w=w, gate=near)
    moe_norm_block(far, far, *b, pre_w=w, gate=far)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o = [t.as_strided((n, 2, d // 2), (t.stride(0), d // 2, 1)) for t in (near, far)]
    out = [torch.empty(n, 2, d // 2, dtype=BF, device="cuda") for _ in range(2)]
    for t, r in zip(o, out):
        moe_norm_gated(t, t, w[:d // 2], r)
    assert torch.equal(*out)


@pytest.mark.parametrize("rows", [1023, 1024, 1025, 2500])
def test_norm_rows_on_both_sides_of_the_rule(rows):
    # each row is a row's own: the same as in calls of few rows
    y, h = torch.randn(rows, 2048, device="cuda"), torch.randn(rows, 2048, device="cuda").to(BF)
    w = torch.randn(2048, device="cuda").to(BF)
    ho, x = torch.empty_like(h), torch.empty_like(h)
    moe_norm_block(y, h, ho, x, pre_w=w, post_w=w, gate=h)
    for at in (0, 511, rows - 1):
        r = slice(at, at + 1)
        want = od.norm_block(*(t.double().cpu().numpy() for t in (y[r], h[r], h[r], w, w)), "sigmoid", 1.0, 1e-6, 0.0)
        # one rounding to bf16; before it 2^-19 of the sum's parts, which are below 2^6 here, and of x's below 2^8
        for got, ref, part in ((ho, want[0], 2.0 ** 6), (x, want[1], 2.0 ** 8)):
            assert np.allclose(got[r].double().cpu().numpy(), ref, rtol=2.0 ** -8 * 1.02, atol=2.0 ** -19 * part)


@pytest.mark.parametrize("tokens", [1023, 1024, 1025])
def test_gated_rows_on_both_sides_of_the_rule(tokens):
    o, z = (torch.randn(tokens, 32, 128, device="cuda").to(BF) for _ in range(2))
    w = torch.randn(128, device="cuda").to(BF)
    out = torch.empty_like(o)
    moe_norm_gated(o, z, w, out)
    want = od.norm_gated(*(t.double().cpu().numpy() for t in (o, z, w)), "silu", False, 1e-6, 0.0)
    # one rounding to bf16, and 2^-19 before it
    assert np.allclose(out.double().cpu().numpy(), want, rtol=2.0 ** -8 * 1.02, atol=2.0 ** -24)


@pytest.mark.parametrize("lens,hk,hv", [([9000], 64, 128), ([5000, 6000, 70], 64, 128), ([300] * 40, 64, 128)])
def test_more_chunks_than_the_work_space_holds(lens, hk, hv):
    # the state goes on from one window of chunks (some 125 of these heads) to the next; against the call token by token
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


@pytest.mark.parametrize("lens", [[100, 30, 500, 30, 0, 500, 64, 1], [70] * 128, [70] * 129, [25, 26] * 64])
def test_sequences_in_any_order_of_lengths(lens):
    c = Case(lens, hk=1, hv=1, dk=64, dv=64, seed=len(lens), pad=2)
    c.check(c.forward())


@pytest.mark.parametrize("n", [4, 90])
@pytest.mark.parametrize("first", [5, 64, 100])
def test_rows_before_the_first_sequence(n, first):
    # no sequence holds them: as if the tensors began behind them, and they are left as they were
    c = Case([n, 3], hk=1, hv=2, seed=first, pad=2)
    want = c.forward()
    d = c.device()
    front = lambda t: torch.cat([torch.full_like(t[:1], 7.0).expand(first, *t.shape[1:]), t])
    x = front(c.x)
    d["g"], d["beta"], d["out"] = front(d["g"]), front(d["beta"]), front(d["out"])
    d["cu"] += first
    q, k, v = c.views(x)
    c.op.moe_delta_forward(q, k, v, **d)
    c.op.moe_delta_sync()
    # (a chunk's tokens are the sequence's own, wherever it begins)
    assert torch.equal(d["out"][first:], want["out"]) and (d["out"][:first] == 7.0).all()
    assert torch.equal(d["state"], want["state"])


@pytest.mark.parametrize("n", [1, 25])
def test_the_most_sequences(n):
    c = Case([n] * 4096, hk=1, hv=1, dk=64, dv=64, seed=n)
    a, b = c.forward(max_q=n), c.forward(max_q=1)
    c.op.moe_delta_sync()
    for s in (0, 1, 2047, 4095):
        r = slice(n * s, n * s + n)
        q, k, v = c.views(c.x64)
        o, S1, mag, size = od.rule(q[r], k[r], v[r], c.g64[r], c.b64[r], c.st64[c.s_in[s]], c.scale)
        for d in (a, b):
            # the bounds of the rule's own tests
            tol = 2.0 ** -8 * 1.01 * np.abs(o) + 2.0 ** -10 * mag + 2.0 ** -17 * (mag + c.scale * size) + 2.0 ** -24
            assert (np.abs(d["out"][r].double().cpu().numpy() - o) <= tol).all()
            off = np.sqrt(((d["state"][c.s_out[s]].double().cpu().numpy() - S1) ** 2).sum(1))
            assert (off <= 2.0 ** -17 * size[-1] + 2.0 ** -40).all()


@pytest.mark.parametrize("n", [3, 80])
def test_a_state_that_two_sequences_begin_from(n):
    c = Case([n, n + 1], seed=n, keep=(0, 1))
    c.s_in[1] = c.s_in[0]
    c.check(c.forward())
    c.op.moe_delta_sync()


def test_a_cut_sequence_that_is_longer_than_the_work_space():
    # 313 chunks of 64 heads: cut in each of two windows, the state goes on from one to the other
    c = Case([20000], hk=32, hv=64, dk=64, dv=64, seed=3, decay=0.003)
    a, b = c.forward(max_q=1), c.forward()
    torch.cuda.synchronize()
    x, y = (d["state"][c.s_out[0]].double() for d in (a, b))
    # as above: far above what rounding makes of either, far below a chunk that is missing
    assert ((x - y).norm(dim=1) <= 2.0 ** -13 * x.norm(dim=1) + 1e-6).all()
    x, y = a["out"].double(), b["out"].double()
    assert ((x - y).norm(dim=2) <= 2.0 ** -6 * x.norm(dim=2) + 1e-6).all()
    c.op.moe_delta_sync()


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from delta_helpers import Case
from expert_cached_decode_gb300 import moe_norm_block, moe_norm_gated
c = Case([2000, 1, 70], hk=1, hv=2, seed=1)
d = c.device()
w = torch.ones(128, dtype=c.dtype, device="cuda")
out, h, x = torch.empty_like(d["out"]), torch.empty_like(d["out"]).view(-1, 128), torch.empty_like(d["out"]).view(-1, 128)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    c.forward(d)
    moe_norm_gated(d["out"], d["out"], w, out)
    moe_norm_block(out.view(-1, 128), None, h, x, pre_w=w)
graph.replay()
c.check(d)
c.op.moe_delta_sync()
"""


def test_the_first_call_of_a_process_is_captured():
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
