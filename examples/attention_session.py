"""A serving session of one decoder layer: attention over a paged int8 cache
next to the routed-expert FFN.

Two sequences are answered together.  Their prompts go through in one ragged
call, then each step appends one token per sequence.  Every step adds up what
attention gave to each cell, and when a sequence would pass `limit` cells the
ones of the least weight leave: the kept cells move to the other half of the
page pool and the step goes on there.  The single-token step is captured once
in a CUDA graph and replayed, also after an eviction: lengths, positions and
page tables are device memory that the replay reads.

    python examples/attention_session.py        # needs the GPU and the built library

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

from expert_cached_decode_gb300 import PagedAttention, Rope  # noqa: E402


def tiny_experts():
    """The tiny routed-expert layer of the synthetic workloads, every expert resident."""
    from expert_cached_decode_gb300 import MoELayer
    from moe_inputs import synth
    s = synth(1)
    wl = s.wl
    pool = torch.empty((wl.keys, s.B), dtype=torch.uint8, pin_memory=True)
    for e in range(wl.keys):
        pool[e] = torch.from_numpy(s.expert_packed(e))
    bits, _, bias = s.router(0)
    layer = MoELayer(wl.d, wl.f, wl.n_experts, wl.top_k, 1, bits.reshape(1, wl.n_experts, wl.d), bias.reshape(1, -1),
                     np.stack([s.shared_packed(0)]), pool)
    layer.moe_cache_configure(wl.capacity, np.arange(wl.keys))
    return layer


class Session:
    """hidden = d; every sequence holds at most `limit` cells and is brought down to `budget` before it would pass that."""

    def __init__(self, experts, d=256, n_seqs=2, limit=512, budget=256, recent=64, n_q_heads=8, n_kv_heads=2, head_dim=64,
                 page_cells=16, kv_dtype=torch.int8, decay=1.0, seed=0):
        dev = "cuda"
        self.experts, self.d, self.n, self.decay = experts, d, n_seqs, decay
        self.limit, self.budget, self.recent = limit, budget, recent
        self.hq, self.hkv, self.hd = n_q_heads, n_kv_heads, head_dim
        self.att = PagedAttention(n_q_heads, n_kv_heads, head_dim, page_cells, kv_dtype=kv_dtype,
                                  rope=Rope(head_dim, base=1e6, scaling="yarn", factor=4.0, original_len=32768))
        per = -(-limit // page_cells)
        # two halves of the pool: an eviction reads one and writes the other
        order = torch.from_numpy(np.random.default_rng(seed).permutation(2 * n_seqs * per).astype(np.int32)).to(dev)
        self.halves = list(order.reshape(2, n_seqs, per))
        self.table = self.halves[0].clone()
        self.cells = torch.zeros((2 * n_seqs * per, page_cells, self.att.cell_bytes), dtype=torch.uint8, device=dev)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=dev)       # cells, read on the GPU
        self.pos = torch.zeros(n_seqs, dtype=torch.int32, device=dev)        # positions: go on when cells leave
        self.host_lens = [0] * n_seqs
        self.acc = torch.zeros((n_seqs, per * page_cells), device=dev)       # weight of each cell so far
        self.keep = torch.zeros((n_seqs, budget), dtype=torch.int32, device=dev)
        self.new_lens, self.kept_acc = torch.zeros_like(self.lens), torch.zeros((n_seqs, budget), device=dev)
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).to(torch.bfloat16).to(dev)
        self.w_qkv, self.w_o = rand(d, (n_q_heads + 2 * n_kv_heads) * head_dim), rand(n_q_heads * head_dim, d)
        self.one_each = torch.arange(n_seqs + 1, dtype=torch.int32, device=dev)
        self.x = torch.zeros((n_seqs, d), dtype=torch.bfloat16, device=dev)  # input of the next single-token step
        self.graph, self.evictions = None, 0
        self.warm = False                        # one eager step goes before the capture

    def _layer(self, x, positions, cu_q, max_q):
        """The layer on x [tokens, d]; the last call's q, attention and lse stay in self for a look."""
        n = x.shape[0]
        qkv = (x @ self.w_qkv).view(n, -1, self.hd)
        q, k, v = qkv.split([self.hq, self.hkv, self.hkv], 1)                # slices of one projection, as they are
        self.q = torch.empty((n, self.hq, self.hd), dtype=x.dtype, device=x.device)
        self.o = torch.empty_like(self.q)
        self.lse = torch.empty((n, self.hq), device=x.device)
        self.att.moe_attn_append(self.cells, q, k, v, positions, cu_q, self.lens, self.table, self.q)
        self.att.moe_attn_forward(self.cells, self.q, cu_q, self.lens, self.table, self.o, self.lse, max_q=max_q)
        self.att.moe_attn_weights(self.cells, self.q, self.lse, cu_q, self.lens, self.table, self.acc, self.acc,
                                  decay=self.decay, max_q=max_q)
        h = x + self.o.view(n, -1) @ self.w_o
        y = torch.empty((n, self.d), device=x.device)
        self.experts.moe_forward(0, h, y)
        z = h.float() + y
        return (z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def prompt(self, prompts):
        """prompts: per sequence [tokens, d] bf16 (device); one ragged call."""
        n = [p.shape[0] for p in prompts]
        if max(n) > self.limit:
            raise ValueError("a prompt is longer than a sequence may be")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        pos = torch.cat([torch.arange(k, dtype=torch.int32) for k in n]).cuda()
        self.lens.copy_(torch.tensor(n, dtype=torch.int32))
        self.pos.copy_(self.lens)
        self.host_lens = list(n)
        out = self._layer(torch.cat(prompts), pos, cu, max(n))
        self.x.copy_(out[(cu[1:] - 1).long()])

    def _step(self):
        self.lens += 1
        self.x.copy_(self._layer(self.x, self.pos, self.one_each, 1))
        self.pos += 1

    def step(self, graph=True):
        """One token of every sequence."""
        if max(self.host_lens) + 1 > self.limit:
            self.evict()
        if graph and self.graph is None and self.warm:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._step()
        if graph and self.graph is not None:
            self.graph.replay()
        else:
            self._step()
            self.warm = True
        self.host_lens = [k + 1 for k in self.host_lens]

    def evict(self):
        old, new = self.halves
        self.att.moe_attn_evict(self.cells, self.acc, self.lens, self.table, self.recent, new, self.keep, self.new_lens,
                                self.kept_acc)
        self.halves = [new, old]
        self.table.copy_(new)
        self.lens.copy_(self.new_lens)
        self.acc.zero_()
        self.acc[:, :self.budget] = self.kept_acc
        self.host_lens = [min(k, self.budget) for k in self.host_lens]
        self.evictions += 1


def main():
    experts = tiny_experts()
    s = Session(experts)
    g = torch.Generator().manual_seed(1)
    s.prompt([torch.randn(n, s.d, generator=g).to(torch.bfloat16).cuda() for n in (400, 150)])
    for _ in range(4):
        s.step()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(500):
        s.step()
    end.record()
    s.att.moe_attn_sync()                     # raises if a page or a length was out of range on the GPU
    experts.moe_sync()
    print(f"{start.elapsed_time(end) * 1e3 / 500:.1f} us per step of {s.n} tokens, {s.evictions} evictions, "
          f"cells now {s.host_lens}, positions {s.pos.tolist()}")


if __name__ == "__main__":
    main()
