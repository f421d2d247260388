"""The gated delta rule, its convolution and gates, the norms and the routed
experts together, as the example runs them: captured steps against eager ones,
sequences that come and go, and each call of a prompt and of a step against the
64-bit oracle over what it was given."""

import numpy as np
import pytest
import torch

from delta_helpers import unit
from oracle import delta as od

pytestmark = pytest.mark.gpu

IN = 2.0 ** -19             # fp32 sums and a fast exponential, relative to the result and to the parts of a sum


def _f(t):
    return t.double().cpu().numpy()


def _check_calls(s, cu, slots_in, slots_out, state, conv):
    """s.last against the oracle; state, conv: before the call."""
    torch.cuda.synchronize()
    t = {k: _f(v) for k, v in s.last.items()}
    u = unit(torch.bfloat16) * 1.01
    near = lambda got, want, part=0.0: np.testing.assert_array_less(np.abs(got - want), (u + IN) * np.abs(want) + IN * part + 2.0 ** -23)
    state, conv = _f(state), _f(conv)
    want_state, want_conv = state.copy(), conv.copy()
    n = t["x"].shape[0]
    for i in range(len(cu) - 1):
        r = slice(cu[i], cu[i + 1])
        old = conv[slots_in[i]] if slots_in[i] >= 0 else np.zeros_like(conv[0])
        y, new, mag = od.conv(t["qkv"][r], _f(s.conv_w), _f(s.conv_bias), old)
        near(t["y"][r], y, mag)
        S0 = state[slots_in[i]] if slots_in[i] >= 0 else np.zeros_like(state[0])
        o, S1, mag, size = od.rule(t["q"][r], t["k"][r], t["v"][r], t["g"][r], t["beta"][r], S0, s.dk ** -0.5)
        # the bounds of the rule's own tests: 2^-17 of what goes into a column, 2^-10 of the outputs' own products
        assert (np.abs(t["o"][r] - o) <= u * np.abs(o) + 2.0 ** -10 * mag + 2.0 ** -17 * (mag + s.dk ** -0.5 * size) + 2.0 ** -24).all()
        if slots_out[i] >= 0:
            got = _f(s.state[slots_out[i]])
            assert (np.sqrt(((got - S1) ** 2).sum(1)) <= 2.0 ** -17 * size[-1] + 2.0 ** -40).all()
            want_state[slots_out[i]], want_conv[slots_out[i]] = got, new
    assert np.array_equal(_f(s.state), want_state) and np.array_equal(_f(s.conv_state), want_conv)
    g, beta = od.gates(t["a"], t["b"], _f(s.a_log), _f(s.dt_bias))
    assert np.allclose(t["g"], g, rtol=2.0 ** -20, atol=2.0 ** -40) and np.allclose(t["beta"], beta, rtol=2.0 ** -20, atol=0)
    near(t["gated"], od.norm_gated(t["o"], t["z"].reshape(n, s.hv, s.dv), _f(s.head_w), "silu", False, 1e-6, 0.0))
    h, x = od.norm_block(t["mixed"], t["x"], None, None, _f(s.ffn_w), "none", 1.0, 1e-6, 0.0)
    part = np.abs(t["mixed"]) + np.abs(t["x"])
    near(t["h"], h, part)
    near(t["ffn_in"], x, part / np.sqrt((h * h).mean(-1, keepdims=True) + 1e-6))
    h, x = od.norm_block(t["ffn"], t["h"], None, None, _f(s.next_w), "none", 1.0, 1e-6, 0.0)
    near(t["out"], x, (np.abs(t["ffn"]) + np.abs(t["h"])) / np.sqrt((h * h).mean(-1, keepdims=True) + 1e-6))


def _run(experts, graph):
    from examples.delta_session import Session
    s = Session(experts)
    g = torch.Generator().manual_seed(3)
    prompt = lambda n: torch.randn(n, s.d, generator=g).to(torch.bfloat16).cuda()
    state, conv = s.state.clone(), s.conv_state.clone()
    s.prompt([0, 1, 2], [3, 0, 2], [prompt(n) for n in (90, 31, 1)])
    _check_calls(s, [0, 90, 121, 122], [-1] * 3, [3, 0, 2], state, conv)
    outs = []
    for i in range(30):
        if i == 12:
            s.end(1)
        if i == 20:
            s.prompt([1], [4], [prompt(70)])
        kept = s.state[0].clone()
        s.step(graph=graph)
        outs.append(s.x.clone())
        if 12 <= i:
            assert torch.equal(s.state[0], kept)             # nobody's any more
    s.rule.moe_delta_sync()
    return s, torch.stack(outs)


def test_a_session():
    from examples.attention_session import tiny_experts
    experts = tiny_experts()
    eager, a = _run(experts, False)
    graphed, b = _run(experts, True)
    assert graphed.graph is not None
    assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    assert torch.equal(eager.state, graphed.state) and torch.equal(eager.conv_state, graphed.conv_state)
    s = eager
    state, conv, slots = s.state.clone(), s.conv_state.clone(), s.slots.tolist()
    assert slots == [3, 4, 2]
    s.x = s.x.clone()                                        # (the step writes its outputs over its inputs)
    s.last = None
    x = s.x.clone()
    s._layer(x, s.one_each, s.slots, s.slots, 1)
    _check_calls(s, [0, 1, 2, 3], slots, slots, state, conv)
    experts.close()
