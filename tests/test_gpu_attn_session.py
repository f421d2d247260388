"""The attention operators and the routed experts together, as the example
runs them: captured steps against eager ones, evictions, and a step's
attention against the oracle over what the cache then holds."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu


def _run(experts, graph, kv_dtype, steps=60):
    from examples.attention_session import Session
    s = Session(experts, limit=96, budget=48, recent=16, kv_dtype=kv_dtype)
    g = torch.Generator().manual_seed(3)
    s.prompt([torch.randn(n, s.d, generator=g).to(torch.bfloat16).cuda() for n in (90, 31)])
    outs = []
    for _ in range(steps):
        s.step(graph=graph)
        outs.append(s.x.clone())
    s.att.moe_attn_sync()
    return s, torch.stack(outs)


@pytest.mark.parametrize("kv_dtype", [torch.int8, torch.bfloat16])
def test_a_session(kv_dtype):
    from examples.attention_session import tiny_experts
    experts = tiny_experts()
    eager, a = _run(experts, False, kv_dtype)
    graphed, b = _run(experts, True, kv_dtype)
    assert graphed.graph is not None and graphed.evictions == 2 == eager.evictions
    assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    s = graphed
    assert s.lens.tolist() == s.host_lens and s.pos.tolist() == [150, 91]
    # every cell of the cache back as values, and the last step's attention and weights from those
    lens = s.host_lens
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((sum(lens), s.hkv, s.hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s.att.moe_attn_read(s.cells, cu, s.lens, s.table, k, v)
    s.att.moe_attn_sync()
    at = np.concatenate([[0], np.cumsum(lens)])
    for i in range(s.n):
        k64, v64 = (t[at[i]:at[i + 1]].double().cpu().numpy() for t in (k, v))
        want, lse, mag = oa.attention(s.q[i:i + 1].double().cpu().numpy(), k64, v64, 0, s.hd ** -0.5)
        got = s.o[i:i + 1].double().cpu().numpy()
        # the read rounds a cell's values to bf16, once (int8 cells): 2^-8 of |q||k| in a score, of |v| in a sum;
        # the probabilities' and the output's roundings are 2^-8 of sum p|v| and of |out|
        q64 = s.q[i].double().cpu().numpy()
        span = 2.0 ** -8 * max(np.abs(q64[h]) @ np.abs(k64[:, h // (s.hq // s.hkv)]).max(0) for h in range(s.hq)) * s.hd ** -0.5
        tol = (2 * np.expm1(span) + 3 * 2.0 ** -8) * mag + 1e-6
        assert (np.abs(got - want) <= tol).all()
        assert np.abs(s.lse[i].cpu().numpy() - lse[0]).max() <= span + 1e-4
        # what is summed up is one per head and token, less what left with evicted cells
        total = float(s.acc[i, :lens[i]].double().sum())
        assert 0 < total <= s.hq * int(s.pos[i]) * (1 + 1e-3)
        assert not s.acc[i, lens[i]:].any()
    experts.close()
