"""Cases of the attention side of the serving engine: the paged KV cache, the
rotation and write of new cells, attention over the pages, and eviction by
accumulated attention weight.

A cell holds the K and V vectors of one token for every K/V head,
[K heads][V heads] in 16 bits, or int8 codes followed by one fp32 scale per
head vector ([K scales][V scales]), padded to 16 bytes; 4 heads of 128 give
the int8 cell of 1,056 bytes.  A page is `page` cells; a sequence's pages are
in its row of the block table.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}
ROPE_BASE = 1e6
YARN = dict(factor=4.0, original_len=32768, beta_fast=32.0, beta_slow=1.0)


# ------------------------------------------------------------------- cases --
def _case(op, **kw):
    c = dict(op=op, seqs=1, q=1, kv=4096, spread=1, mixed=False, hq=32, hkv=4, d=128, page=32, cache="bf16", io="bf16",
             window=0, rot=0, interleaved=False, scaling="none", budget=0, recent=0)
    c.update(kw)
    return c


def listed():
    return [
        # the step of 16 running sequences: rotate the new token's q and k, write int8 cells, read the cells back
        dict(_case("append", seqs=16, kv=8192, spread=16, cache="int8", rot=128), name="append_step"),
        # a prefill chunk at the end of a 131,072-cell context, YaRN, a part of the head rotated in the interleaved layout
        dict(_case("append", q=12288, kv=131072, rot=64, interleaved=True, scaling="yarn"), name="append_chunk"),
        # the first tokens of an answer: one token, a short prompt; latency
        dict(_case("forward", kv=300, hq=16, hkv=2, page=16), name="token_short"),
        # one token over a full context of int8 cells: the work has to be split along the cache
        dict(_case("forward", kv=131072, cache="int8"), name="token_long"),
        # a step of 32 sequences of very different lengths
        dict(_case("forward", seqs=32, kv=16384, spread=16), name="tokens_ragged"),
        # verification of five drafted tokens for eight sequences over int8 cells
        dict(_case("forward", seqs=8, q=5, kv=32768, spread=4, cache="int8"), name="verify"),
        # a step that mixes one prompt's chunk with single tokens of 15 others; smaller heads, a window
        dict(_case("forward", seqs=16, q=1000, kv=8192, spread=3, mixed=True, hq=24, hkv=8, d=64, page=64, cache="fp16",
                   io="fp16", window=4096), name="mixed"),
        # a prefill chunk at the end of a long prompt: the tensor cores' work
        dict(_case("forward", q=4096, kv=32768), name="chunk"),
        # the weights that one token's attention gives to the cells of four int8 sequences
        dict(_case("weights", seqs=4, kv=65536, spread=4, cache="int8"), name="weights_step"),
        # the weights that a chunk's attention gives
        dict(_case("weights", q=1024, kv=16384), name="weights_chunk"),
        # a full context brought down to the cells that stay in device memory
        dict(_case("evict", kv=131072, cache="int8", budget=32768, recent=1024), name="evict_long"),
        # several sequences over their budget at once, one below it
        dict(_case("evict", seqs=12, kv=6000, spread=8, budget=1500, recent=64, page=16, hkv=2), name="evict_ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "forward", "forward", "forward", "weights", "evict"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 6, 8])
    io = rng.choice(["bf16", "bf16", "fp16"])
    c = _case(op, d=d, hkv=hkv, hq=hq, page=rng.choice([1, 16, 24, 32, 64, 128]), io=io, cache=rng.choice([io, "int8"]))
    c["spread"] = rng.choice([1, 3, 16])
    if op == "append":
        c.update(seqs=_log(rng, 1, 64), q=_log(rng, 1, 256), rot=rng.choice([d, d, d // 2, d // 4]),
                 interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
        c["kv"] = c["q"] + _log(rng, 16, 8192)
    elif op == "evict":
        c.update(seqs=_log(rng, 1, 8), kv=_log(rng, 64, 65536))
        c["budget"] = max(1, int(c["kv"] * rng.uniform(0.05, 0.9)))
        c["recent"] = rng.randint(0, c["budget"])
    else:
        c.update(seqs=_log(rng, 1, 32), kv=_log(rng, 64, 65536), q=rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, 2048)]))
        c["q"] = min(c["q"], c["kv"])
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
        c["mixed"] = c["q"] > 16 and rng.random() < 0.3
        while c["seqs"] * c["q"] * c["kv"] * c["hq"] > 4096 * 32768 * 8 or c["seqs"] * c["kv"] > 1 << 20:
            if c["seqs"] > 1:
                c["seqs"] = (c["seqs"] + 1) // 2
            else:
                c["kv"] //= 2
            c["q"] = min(c["q"], c["kv"])
    return c


def _lens(c):
    """(new tokens, cells) of each sequence: the lengths fall from kv to about kv / spread."""
    n = c["seqs"]
    kv = [max(1, round(c["kv"] * c["spread"] ** (-i / max(1, n - 1))) - (i * 7 % 13 if i else 0)) for i in range(n)]
    q = [min(c["q"] if i == 0 or not c["mixed"] else 1, kv[i]) for i in range(n)]
    return q, kv


def _pairs(c):
    """(row, cell) pairs that are visible, for one head."""
    w = c["window"]
    total = 0
    for q, kv in zip(*_lens(c)):
        first, last = kv - q + 1, kv                     # cells seen by the first and the last row
        if not w or last <= w:
            total += (first + last) * q // 2
        elif first >= w:
            total += w * q
        else:
            total += (first + w) * (w - first + 1) // 2 + (last - w) * w
    return total


def _cells_read(c):
    """Cells that some row of the call sees."""
    return sum(kv if not c["window"] else min(kv, c["window"] + q - 1) for q, kv in zip(*_lens(c)))


def _cell_data(c):
    """Bytes of a cell that carry something."""
    vec = 2 * c["hkv"] * c["d"]
    return vec + 8 * c["hkv"] if c["cache"] == "int8" else 2 * vec


def work(c):
    q, kv = _lens(c)
    tokens, rows, heads = sum(q), sum(q) * c["hq"], c["hkv"] * c["d"]
    if c["op"] == "append":
        values = 4 * tokens * heads if c["cache"] == "int8" else 0
        return {"bytes": 4 * rows * c["d"] + 4 * tokens * heads + tokens * _cell_data(c) + values,
                "flops": 3 * tokens * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "forward":
        return {"bytes": 4 * rows * c["d"] + 4 * rows + _cells_read(c) * _cell_data(c), "flops": 4 * c["d"] * c["hq"] * _pairs(c)}
    if c["op"] == "weights":
        return {"bytes": 2 * rows * c["d"] + 4 * rows + _cells_read(c) * _cell_data(c) // 2 + 8 * sum(kv),
                "flops": 2 * c["d"] * c["hq"] * _pairs(c)}
    kept = sum(min(n, c["budget"]) for n in kv)
    return {"bytes": 4 * sum(kv) + 8 * kept + 2 * kept * _cell_data(c), "flops": 0}


# ------------------------------------------------------------------ inputs --
def _cell_bytes(c):
    return (_cell_data(c) + 15) // 16 * 16


def _turns(c):
    """Turns per position of each rotated pair, and the factor on cosine and sine (64 bits)."""
    rot, s = c["rot"], c["scaling"]
    i = np.arange(rot // 2, dtype=np.float64)
    base = ROPE_BASE * (YARN["factor"] ** (rot / max(1, rot - 2)) if s == "ntk" else 1.0)
    f = base ** (-2.0 * i / rot)
    if s == "linear":
        f = f / YARN["factor"]
    if s == "yarn":
        def dim(turns):
            return rot * math.log(YARN["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))
        low, high = max(0, math.floor(dim(YARN["beta_fast"]))), min(rot - 1, math.ceil(dim(YARN["beta_slow"])))
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0, 1)
        f = f * (1 - ramp) + f / YARN["factor"] * ramp
    return f / (2 * math.pi), 0.1 * math.log(YARN["factor"]) + 1.0 if s == "yarn" else 1.0


def _quantised(x):
    """Head vectors x[..., D] as int8 codes and fp32 scales, absmax / 127."""
    top = x.abs().amax(-1, keepdim=True)
    codes = torch.round(x * torch.where(top > 0, 127.0 / top, 0.0))
    return codes.to(torch.int8), top / 127.0


def _packed(c, k, v):
    """Cells [N, cell_bytes] of K and V vectors [N, hkv, D]."""
    n = k.shape[0]
    if c["cache"] != "int8":
        return torch.stack([k, v], 1).to(DTYPES[c["cache"]]).reshape(n, -1).view(torch.uint8)
    (kc, ks), (vc, vs) = _quantised(k.float()), _quantised(v.float())
    raw = torch.cat([torch.stack([kc, vc], 1).reshape(n, -1).view(torch.uint8),
                     torch.stack([ks, vs], 1).reshape(n, -1).view(torch.uint8)], 1)
    return torch.nn.functional.pad(raw, (0, _cell_bytes(c) - raw.shape[1]))


def _values(c, cells, dtype=torch.float32):
    """K and V vectors [..., hkv, D] that cells [..., cell_bytes] stand for."""
    h, d, lead = c["hkv"], c["d"], cells.shape[:-1]
    if c["cache"] != "int8":
        kv = cells.view(DTYPES[c["cache"]]).reshape(*lead, 2, h, d).to(dtype)
    else:
        codes = cells[..., :2 * h * d].view(torch.int8).reshape(*lead, 2, h, d)
        scales = cells[..., 2 * h * d:2 * h * d + 8 * h].contiguous().view(torch.float32).reshape(*lead, 2, h, 1)
        kv = codes.to(dtype) * scales.to(dtype)
    return kv[..., 0, :, :], kv[..., 1, :, :]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.default_rng(seed)
    q_lens, kv_lens = _lens(c)
    n, page, tokens, io = c["seqs"], c["page"], sum(q_lens), DTYPES[c["io"]]
    need = [-(-kv // page) for kv in kv_lens]
    kept = [-(-min(kv, c["budget"]) // page) for kv in kv_lens] if c["op"] == "evict" else [0] * n
    n_pages = sum(need) + sum(kept) + 2
    order = host.permutation(n_pages).astype(np.int32)
    ends, ends_kept = np.cumsum(need), sum(need) + np.cumsum(kept)
    table = np.zeros((n, max(need)), np.int32)
    table_kept = np.zeros((n, max(max(kept), 1)), np.int32)
    for i in range(n):
        table[i, :need[i]] = order[ends[i] - need[i]:ends[i]]
        table_kept[i, :kept[i]] = order[ends_kept[i] - kept[i]:ends_kept[i]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    st = {"c": c, "dtype": io, "n_pages": n_pages, "max_q": max(q_lens), "max_kv": max(kv_lens),
          "cu_q": torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda"),
          "kv_lens": torch.tensor(kv_lens, dtype=torch.int32, device="cuda"),
          "table": torch.from_numpy(table).cuda(), "scale": c["d"] ** -0.5}
    if c["op"] == "append":
        st["cells"] = torch.zeros((n_pages, page, _cell_bytes(c)), dtype=torch.uint8, device="cuda")
        # q, k and v as the fused projection leaves them, one row per token
        heads = (c["hq"] + 2 * c["hkv"])
        qkv = normal(tokens, heads, c["d"]).to(io)
        st["q"], st["k"], st["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], 1)
        st["positions"] = torch.cat([torch.arange(kv - q, kv) for q, kv in zip(q_lens, kv_lens)]).to(torch.int32).cuda()
        turns, st["factor"] = _turns(c)
        st["turns"] = torch.from_numpy(np.round(turns * 2.0 ** 64).astype(np.uint64).view(np.int64)).cuda()
        st["q_out"] = torch.empty((tokens, c["hq"], c["d"]), dtype=io, device="cuda")
        st["k_out"], st["v_out"] = (torch.empty((tokens, c["hkv"], c["d"]), dtype=io, device="cuda") for _ in range(2))
    else:
        # cells with the keys' usual spread: channels of different size, a first cell that draws weight
        k = normal(n_pages * page, c["hkv"], c["d"]) * (0.5 + 1.5 * torch.rand(c["hkv"], c["d"], generator=g, device="cuda"))
        v = normal(n_pages * page, c["hkv"], c["d"])
        st["cells"] = _packed(c, k, v).reshape(n_pages, page, -1)
        del k, v
        st["q"] = normal(tokens, c["hq"], c["d"], std=1.5).to(io)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((tokens, c["hq"]), dtype=torch.float32, device="cuda")
    if c["op"] == "weights":
        st["lse"] = _forward(st)[1]
        st["acc"] = torch.rand(n, max(kv_lens), generator=g, device="cuda").square() * 4
        st["acc_out"] = torch.zeros_like(st["acc"])
        st["decay"] = 0.96875
    if c["op"] == "evict":
        # many cells that hardly any row looked at (ties at few values), few that most did
        acc = torch.exp2(torch.randint(-12, 0, (n, max(kv_lens)), generator=g, device="cuda").float())
        heavy = torch.rand(acc.shape, generator=g, device="cuda")
        st["acc"] = torch.where(heavy < 0.2, heavy * 40, acc)
        st["table_kept"] = torch.from_numpy(table_kept).cuda()
        st["keep"] = torch.empty((n, c["budget"]), dtype=torch.int32, device="cuda")
        st["lens_kept"] = torch.empty(n, dtype=torch.int32, device="cuda")
        st["acc_kept"] = torch.empty((n, c["budget"]), dtype=torch.float32, device="cuda")
    if own:
        from expert_cached_decode_gb300.attention import PagedAttention, Rope
        rope = None
        if c["op"] == "append":
            rope = Rope(c["rot"], base=ROPE_BASE, interleaved=c["interleaved"], scaling=c["scaling"], **YARN)
        st["att"] = PagedAttention(c["hq"], c["hkv"], c["d"], page, kv_dtype=DTYPES[c["cache"]], dtype=io,
                                   window=c["window"], rope=rope)
    return st


# -------------------------------------------------------------- plain form --
def _row_index(st):
    """Padded rows: token of row (s, i), whether it exists, and its place in the cache."""
    i = torch.arange(st["max_q"], device="cuda")
    first, n_q = st["cu_q"][:-1, None].long(), st["cu_q"].diff()[:, None]
    token = (first + i).clamp(max=st["q"].shape[0] - 1)
    return token, i < n_q, st["kv_lens"][:, None] - n_q + i


def _scores(st):
    """Scaled scores [n, hkv, G * max_q, kv] with the hidden ones at -inf, and the cells' K and V."""
    c = st["c"]
    token, real, place = _row_index(st)
    n, mq, h, d = c["seqs"], st["max_q"], c["hkv"], c["d"]
    pages = -(-st["max_kv"] // c["page"])
    cells = st["cells"][st["table"][:, :pages].long()].reshape(n, pages * c["page"], -1)[:, :st["max_kv"]]
    k, v = (x.transpose(1, 2) for x in _values(c, cells))                       # [n, hkv, kv, D]
    q = st["q"][token].float().reshape(n, mq, h, -1, d).permute(0, 2, 3, 1, 4)    # [n, hkv, G, max_q, D]
    s = torch.matmul(q.reshape(n, h, -1, d), k.transpose(2, 3)) * st["scale"]
    j = torch.arange(st["max_kv"], device="cuda")
    seen = real[:, :, None] & (j <= place[:, :, None])
    if c["window"]:
        seen &= j > place[:, :, None] - c["window"]
    s.view(n, h, -1, mq, st["max_kv"]).masked_fill_(~seen[:, None, None], -math.inf)
    return s, v, token, real


def _rows(x, st, token, real):
    """Padded [n, hkv, G * max_q, ...] back to [tokens, hq, ...]."""
    c = st["c"]
    x = x.reshape(c["seqs"], c["hq"], st["max_q"], -1).transpose(1, 2)
    return x[real]


def _forward(st):
    s, v, token, real = _scores(st)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + top
    return _rows(o, st, token, real).to(st["dtype"]), _rows(lse, st, token, real)[..., 0]


def _weights(st):
    c = st["c"]
    s, _, token, real = _scores(st)
    lse = st["lse"][token].permute(0, 2, 1).reshape(c["seqs"], c["hkv"], -1, 1)
    p = s.sub_(torch.where(torch.isfinite(lse), lse, math.inf)).exp_()
    out = st["acc"] * st["decay"] + p.sum((1, 2))
    j = torch.arange(st["max_kv"], device="cuda")
    return torch.where(j < st["kv_lens"][:, None], out, 0.0)


def _slots(st):
    """Cell (in the flattened pages) of every token of the call."""
    c, (token, real, place) = st["c"], _row_index(st)
    page = torch.gather(st["table"].long(), 1, place.clamp(min=0).long() // c["page"])
    return (page * c["page"] + place % c["page"])[real]


def _rotated(st, x, dtype=torch.float32):
    c = st["c"]
    half = c["rot"] // 2
    turn = (st["positions"].long()[:, None] * st["turns"]).to(dtype) * 2.0 ** -64       # wraps: the part of a turn
    cos, sin = (f(turn * (2 * math.pi))[:, None] * st["factor"] for f in (torch.cos, torch.sin))
    x = x.to(dtype)
    a, b = (x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]) if c["interleaved"] else (x[..., :half], x[..., half:c["rot"]])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if c["interleaved"] else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., c["rot"]:]], -1)


def _append(st):
    c, slots = st["c"], _slots(st)
    k = _rotated(st, st["k"])
    st["cells"].view(-1, _cell_bytes(c))[slots] = _packed(c, k, st["v"])
    q = _rotated(st, st["q"]).to(st["dtype"])
    if c["cache"] != "int8":
        return {"q": q, "cells": st["cells"].view(DTYPES[c["cache"]])}
    k, v = _values(c, st["cells"].view(-1, _cell_bytes(c))[slots])
    return {"q": q, "k": k.to(st["dtype"]), "v": v.to(st["dtype"])}


def _evict(st):
    c, budget = st["c"], st["c"]["budget"]
    n, lens, acc = c["seqs"], st["kv_lens"][:, None], st["acc"]
    j = torch.arange(acc.shape[1], device="cuda")
    rank = torch.where(torch.isnan(acc), -math.inf, acc)
    # newest cells first, then by weight, then the cells that are not there
    group = torch.where(j >= lens, 0, torch.where(j >= lens - c["recent"], 2, 1))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    order = torch.gather(order, 1, torch.sort(torch.gather(group, 1, order), dim=1, descending=True, stable=True).indices)
    order = torch.nn.functional.pad(order, (0, max(0, budget - order.shape[1])))[:, :budget]
    i = torch.arange(budget, device="cuda")
    new = torch.minimum(lens, torch.full_like(lens, budget))
    keep = torch.sort(torch.where(i < new, order, acc.shape[1]), dim=1).values
    there = i < new
    safe = torch.where(there, keep, 0)
    src = torch.gather(st["table"].long(), 1, safe // c["page"]) * c["page"] + safe % c["page"]
    at = i.expand(n, -1)
    dst = torch.gather(st["table_kept"].long(), 1, torch.where(there, at // c["page"], 0)) * c["page"] + at % c["page"]
    flat = st["cells"].view(-1, _cell_bytes(c))
    flat[dst[there]] = flat[src[there]]
    return {"keep": torch.where(there, keep, -1).int(), "lens": new[:, 0].int(),
            "acc": torch.where(there, torch.gather(acc, 1, safe), 0.0), "cells": st["cells"]}


# -------------------------------------------------------------------- pass --
def run(st):
    op = st["c"]["op"]
    if not own:
        if op == "append":
            return _append(st)
        if op == "forward":
            out, lse = _forward(st)
            return {"out": out, "lse": lse}
        return {"acc": _weights(st)} if op == "weights" else _evict(st)
    att = st["att"]
    if op == "append":
        att.moe_attn_append(st["cells"], st["q"], st["k"], st["v"], st["positions"], st["cu_q"], st["kv_lens"], st["table"],
                            st["q_out"])
        if st["c"]["cache"] != "int8":
            return {"q": st["q_out"], "cells": st["cells"].view(DTYPES[st["c"]["cache"]])}
        att.moe_attn_read(st["cells"], st["cu_q"], st["kv_lens"], st["table"], st["k_out"], st["v_out"])
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    if op == "forward":
        att.moe_attn_forward(st["cells"], st["q"], st["cu_q"], st["kv_lens"], st["table"], st["out"], st["lse"],
                             max_q=st["max_q"], max_kv=st["max_kv"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "weights":
        att.moe_attn_weights(st["cells"], st["q"], st["lse"], st["cu_q"], st["kv_lens"], st["table"], st["acc"],
                             st["acc_out"], decay=st["decay"], max_q=st["max_q"], max_kv=st["max_kv"])
        return {"acc": st["acc_out"]}
    att.moe_attn_evict(st["cells"], st["acc"], st["kv_lens"], st["table"], st["c"]["recent"], st["table_kept"], st["keep"],
                       st["lens_kept"], st["acc_kept"])
    return {"keep": st["keep"], "lens": st["lens_kept"], "acc": st["acc_kept"], "cells": st["cells"]}


# ------------------------------------------------------------------- exact --
def _exact_values(c, cells):
    """K and V [len, hkv, D] in 64 bits from raw cells."""
    h, d = c["hkv"], c["d"]
    if c["cache"] != "int8":
        x = cells.view(DTYPES[c["cache"]]).double().reshape(-1, 2 * h, d)
    else:
        x = cells[:, :2 * h * d].view(torch.int8).double().reshape(-1, 2 * h, d)
        x = x * cells[:, 2 * h * d:2 * h * d + 8 * h].contiguous().view(torch.float32).double()[:, :, None]
    return x[:, :h], x[:, h:]


def _exact_attention(c, st):
    """Row by row of the definition, a sequence and a head at a time: out, lse and the cells' weights."""
    q_lens, kv_lens = _lens(c)
    out, lses, sums = [], [], torch.zeros((c["seqs"], max(kv_lens)), dtype=torch.float64, device="cuda")
    per, t0 = c["hq"] // c["hkv"], 0
    for s, (nq, kv) in enumerate(zip(q_lens, kv_lens)):
        pages = st["table"][s, :-(-kv // c["page"])].long()
        k, v = _exact_values(c, st["cells"][pages].flatten(0, 1)[:kv])
        place = torch.arange(kv - nq, kv, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None]
        hidden = (j > place) | ((j <= place - c["window"]) if c["window"] else torch.zeros_like(j, dtype=torch.bool))
        os, ls = [], []
        for h in range(c["hq"]):
            x = st["q"][t0:t0 + nq, h].double() @ k[:, h // per].T / math.sqrt(c["d"])
            x.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - (lse if c["op"] == "forward" else st["lse"][t0:t0 + nq, h].double())[:, None])
            os.append(p @ v[:, h // per])
            ls.append(lse)
            sums[s, :kv] += p.sum(0)
        out.append(torch.stack(os, 1))
        lses.append(torch.stack(ls, 1))
        t0 += nq
    return torch.cat(out), torch.cat(lses), sums


def exact(c, seed):
    st = prepare(c, seed)
    q_lens, kv_lens = _lens(c)
    if c["op"] == "forward":
        out, lse, _ = _exact_attention(c, st)
        return {"out": out, "lse": lse}
    if c["op"] == "weights":
        sums = _exact_attention(c, st)[2]
        there = torch.arange(max(kv_lens), device="cuda") < st["kv_lens"][:, None]
        return {"acc": torch.where(there, st["decay"] * st["acc"].double() + sums, 0.0)}
    if c["op"] == "evict":
        acc = torch.zeros((c["seqs"], c["budget"]), dtype=torch.float64)
        for s, kv in enumerate(kv_lens):
            a = st["acc"][s, :kv].double().cpu().numpy()
            old = max(0, kv - min(c["recent"], kv))
            room = min(kv, c["budget"]) - (kv - old)
            keep = sorted(sorted(range(old), key=lambda i: (-a[i], i))[:room]) + list(range(old, kv))
            acc[s, :len(keep)] = torch.from_numpy(a[keep])
        return {"keep": None, "lens": None, "acc": acc.cuda(), "cells": None}
    # append: cosine and sine of the angle itself, pair by pair
    turns, factor = _turns(c)
    angle = st["positions"].double()[:, None] * torch.from_numpy(turns).cuda() * (2 * math.pi)
    z = torch.polar(torch.full_like(angle, factor), angle)[:, None]

    def turned(x):
        x = x.double().clone()
        rot = x[..., :c["rot"]]
        at = (slice(0, None, 2), slice(1, None, 2)) if c["interleaved"] else (slice(0, c["rot"] // 2), slice(c["rot"] // 2, None))
        w = torch.complex(rot[..., at[0]].contiguous(), rot[..., at[1]].contiguous()) * z
        rot[..., at[0]], rot[..., at[1]] = w.real, w.imag
        return x

    q, k, v = turned(st["q"]), turned(st["k"]), st["v"].double()
    if c["cache"] == "int8":
        def coded(x):
            scale = x.abs().amax(-1, keepdim=True) / 127
            return torch.round(x / torch.where(scale > 0, scale, 1.0)) * scale
        return {"q": q, "k": coded(k), "v": coded(v)}
    cells = torch.zeros((st["n_pages"] * c["page"], 2, c["hkv"], c["d"]), dtype=torch.float64, device="cuda")
    t = 0
    for s, (nq, kv) in enumerate(zip(q_lens, kv_lens)):
        place = torch.arange(kv - nq, kv, device="cuda")
        at = st["table"][s].long()[place // c["page"]] * c["page"] + place % c["page"]
        cells[at, 0], cells[at, 1] = k[t:t + nq], v[t:t + nq]
        t += nq
    return {"q": q, "cells": cells.reshape(st["n_pages"], c["page"], -1)}
