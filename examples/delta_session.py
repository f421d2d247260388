"""A serving session of one linear-attention layer: the gated delta rule with its
convolution, gates and norms, next to the routed-expert FFN.

Sequences are answered together.  Their prompts go through in one ragged call,
then each step takes one token per sequence.  What a layer keeps of a sequence
has a fixed size: a slot of the rule's state and one of the convolution's last
inputs.  The single-token step is captured once in a CUDA graph and replayed,
also after a sequence has ended or another has taken its place: slots are
device memory that the replay reads.

    python examples/delta_session.py        # needs the GPU and the built library

Weights, prompts and the next token's input (the layer's output, normalised)
are synthetic.
"""

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from examples.attention_session import tiny_experts  # noqa: E402
from expert_cached_decode_gb300 import GatedDelta, moe_norm_block, moe_norm_gated  # noqa: E402


class Session:
    """n_rows sequences at a time; n_slots states, of which row i uses slot self.slots[i] (-1: the row is idle)."""

    def __init__(self, experts, d=256, n_rows=3, n_slots=5, n_k_heads=2, n_v_heads=4, k_dim=64, v_dim=64, taps=4, seed=0):
        self.experts, self.d, self.rows = experts, d, n_rows
        self.hk, self.hv, self.dk, self.dv = n_k_heads, n_v_heads, k_dim, v_dim
        self.rule = GatedDelta(n_k_heads, n_v_heads, k_dim, v_dim, taps=taps)
        dev, C = "cuda", self.rule.channels
        self.state = torch.zeros((n_slots, n_v_heads, k_dim, v_dim), device=dev)
        self.conv_state = torch.zeros((n_slots, taps - 1, C), dtype=torch.bfloat16, device=dev)
        self.slots = torch.full((n_rows,), -1, dtype=torch.int32, device=dev)
        self.one_each = torch.arange(n_rows + 1, dtype=torch.int32, device=dev)
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).to(torch.bfloat16).to(dev)
        self.widths = [C, n_v_heads * v_dim, n_v_heads, n_v_heads]                       # q k v | z | a | b
        self.w_in, self.w_out = rand(d, sum(self.widths)), rand(n_v_heads * v_dim, d)
        self.conv_w, self.conv_bias = rand(taps, C).t().contiguous(), rand(C)
        self.a_log, self.dt_bias = rand(n_v_heads).float(), rand(n_v_heads).float()
        ones = lambda n: torch.ones(n, dtype=torch.bfloat16, device=dev)
        self.head_w, self.ffn_w, self.next_w = ones(v_dim), ones(d), ones(d)
        self.x = torch.zeros((n_rows, d), dtype=torch.bfloat16, device=dev)              # input of the next single-token step
        self.graph, self.warm = None, False

    def _layer(self, x, cu, slots_in, slots_out, max_q):
        """The layer on x [tokens, d] -> its output, normalised.  The call's tensors stay in self.last for a look."""
        n, bf = x.shape[0], torch.bfloat16
        new = lambda *s, dtype=bf: torch.empty(s, dtype=dtype, device=x.device)
        p = x @ self.w_in
        qkv, z, a, b = p.split(self.widths, 1)                                           # slices of one projection, as they are
        y, g, beta = new(n, self.rule.channels), new(n, self.hv, dtype=torch.float32), new(n, self.hv, dtype=torch.float32)
        self.rule.moe_delta_prepare(qkv, self.conv_w, self.conv_bias, self.conv_state, y, a, b, self.a_log, self.dt_bias, g, beta,
                                    cu, slots_in, slots_out)
        nq = self.hk * self.dk
        q, k, v = (t.view(n, -1, w) for t, w in zip(y.split([nq, nq, self.hv * self.dv], 1), (self.dk, self.dk, self.dv)))
        o, gated = new(n, self.hv, self.dv), new(n, self.hv, self.dv)
        self.rule.moe_delta_forward(q, k, v, g, beta, self.state, o, cu, slots_in, slots_out, max_q=max_q)
        moe_norm_gated(o, z.view(n, self.hv, self.dv), self.head_w, gated)
        mixed, h, ffn_in, out = gated.view(n, -1) @ self.w_out, new(n, self.d), new(n, self.d), new(n, self.d)
        moe_norm_block(mixed, x, h, ffn_in, pre_w=self.ffn_w)
        ffn = new(n, self.d, dtype=torch.float32)
        self.experts.moe_forward(0, ffn_in, ffn)
        moe_norm_block(ffn, h, None, out, pre_w=self.next_w)
        self.last = dict(qkv=qkv, a=a, b=b, y=y, q=q, k=k, v=v, g=g, beta=beta, o=o, z=z, gated=gated, mixed=mixed, x=x, h=h,
                         ffn_in=ffn_in, ffn=ffn, out=out)
        return out

    def prompt(self, rows, slots, prompts):
        """New sequences in rows `rows`, their states in slots `slots`; prompts: [tokens, d] bf16 each (device)."""
        n = [p.shape[0] for p in prompts]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        to = torch.tensor(slots, dtype=torch.int32, device="cuda")
        out = self._layer(torch.cat(prompts), cu, torch.full_like(to, -1), to, max(n))   # from zeros
        at = torch.tensor(rows, device="cuda")
        self.x[at] = out[(cu[1:] - 1).long()]
        self.slots[at] = to

    def end(self, row):
        """Row `row` idles: its token is still computed, from zeros, and nothing of it is kept."""
        self.slots[row] = -1

    def _step(self):
        self.x.copy_(self._layer(self.x, self.one_each, self.slots, self.slots, 1))

    def step(self, graph=True):
        """One token of every sequence."""
        if graph and self.graph is None and self.warm:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._step()
        if graph and self.graph is not None:
            self.graph.replay()
        else:
            self._step()
            self.warm = True


def main():
    experts = tiny_experts()
    s = Session(experts)
    g = torch.Generator().manual_seed(1)
    prompt = lambda n: torch.randn(n, s.d, generator=g).to(torch.bfloat16).cuda()
    s.prompt([0, 1, 2], [0, 1, 2], [prompt(n) for n in (400, 150, 3)])
    for _ in range(4):
        s.step()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for i in range(500):
        s.step()
        if i == 250:
            s.end(1)
            s.prompt([1], [4], [prompt(90)])
    end.record()
    s.rule.moe_delta_sync()                   # raises if a slot or an offset was out of range on the GPU
    experts.moe_sync()
    print(f"{start.elapsed_time(end) * 1e3 / 500:.1f} us per step of {s.rows} tokens, slots now {s.slots.tolist()}")


if __name__ == "__main__":
    main()
