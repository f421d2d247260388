"""Cases of the linear-attention layers of the serving engine and of the norms
around its blocks: the short convolution and the gates in front of the gated
delta rule, the rule itself (single tokens, drafts, prompts), the gated norm
behind it, and the norm, gate and residual sum between two blocks.

A call's sequences lie one after another in the rows of its tensors (`cu`:
offsets).  Every sequence has a slot that its state comes from (-1: it starts
from zeros) and one that its state goes to.  q, k and v are slices of one row
per token, [q heads][k heads][v heads].
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------- cases --
def _rule(op, **kw):
    # seqs sequences; the first `long` of them have up to q tokens (evenly spread down to q / spread), the others one
    c = dict(op=op, seqs=1, q=1, spread=1, long=1, hk=16, hv=32, dk=128, dv=128, io="bf16", taps=4, fresh=False,
             keep=False, normalize=True)
    c.update(kw)
    if "long" not in kw:
        c["long"] = c["seqs"]
    return c


def _norm(op, **kw):
    c = dict(op=op, tokens=1, heads=1, d=2048, y="fp32", h="bf16", io="bf16", gate="none", act="sigmoid", post=False,
             pre=True, first=False, offset=0.0, scale=1.0)
    c.update(kw)
    return c


def listed():
    return [
        # one user's answer, a token at a time: latency
        dict(_rule("delta"), name="step_one"),
        # a step of 64 running sequences: the states are read and written once
        dict(_rule("delta", seqs=64), name="step_batch"),
        # drafts of five tokens for eight sequences; the state before them is kept, in case drafts are refused
        dict(_rule("delta", seqs=8, q=5, keep=True), name="verify"),
        # a prefill chunk of one long prompt
        dict(_rule("delta", q=12288, fresh=True), name="chunk"),
        # nine prompts of very different lengths, odd ones among them
        dict(_rule("delta", seqs=9, q=6001, spread=30, fresh=True), name="prompts"),
        # narrow heads: three prompts next to running sequences' single tokens in one call
        dict(_rule("delta", seqs=19, q=1500, spread=3, long=3, hk=8, hv=8, dk=64, dv=64, io="fp16"), name="mixed_narrow"),
        # convolution and gates of a step of 64 sequences
        dict(_rule("prepare", seqs=64), name="prepare_step"),
        # and of a prefill chunk
        dict(_rule("prepare", q=12288, fresh=True), name="prepare_chunk"),
        # the norm behind the rule, gated by a projection: a step of 16 sequences
        dict(_norm("gated", tokens=16, heads=32, d=128, act="silu"), name="gated_step"),
        # and a prefill chunk
        dict(_norm("gated", tokens=12288, heads=32, d=128, act="silu"), name="gated_chunk"),
        # from the experts' fp32 output to the next block's input, five tokens: latency
        dict(_norm("block", tokens=5), name="block_step"),
        # a prefill chunk, the block's output normed and gated before it joins the residual stream
        dict(_norm("block", tokens=12288, y="bf16", h="fp32", gate="full", post=True, scale=0.5, offset=1.0), name="block_chunk"),
    ]


def draw(rng):
    spread = lambda lo, hi: max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))
    op = rng.choice(("delta", "delta", "delta", "prepare", "gated", "block"))
    io = rng.choice(("bf16", "bf16", "fp16"))
    if op in ("delta", "prepare"):
        hk = rng.choice((1, 2, 3, 4, 8, 16))
        hv = hk * rng.choice((1, 2, 4) if hk <= 8 else (1, 2))
        kind = rng.choice(("step", "drafts", "prompts", "mixed"))
        c = _rule(op, hk=hk, hv=hv, dk=rng.choice((64, 128)), dv=rng.choice((64, 128)), io=io, taps=rng.choice((2, 3, 4)),
                  normalize=rng.random() < 0.8)
        if kind == "step":
            c.update(seqs=spread(1, 64), q=1)
        elif kind == "drafts":
            c.update(seqs=spread(1, 32), q=rng.randint(2, 9), spread=rng.choice((1, 2)), keep=rng.random() < 0.5)
        elif kind == "prompts":
            n = spread(1, 12)
            c.update(seqs=n, q=spread(17, 9000 // n), spread=rng.choice((1, 2, 9)), fresh=rng.random() < 0.7)
        else:
            c.update(seqs=rng.randint(4, 24), q=spread(10, 2500), long=rng.randint(1, 3), spread=rng.choice((1, 3)))
        if kind != "mixed":
            c["long"] = c["seqs"]
        return c
    if op == "gated":
        return _norm("gated", tokens=spread(1, 9000), heads=rng.choice((1, 4, 5, 16, 32)), d=rng.choice((64, 128, 256)), io=io,
                     act=rng.choice(("silu", "sigmoid")), first=rng.random() < 0.3, offset=rng.choice((0.0, 1.0)))
    return _norm("block", tokens=spread(1, 9000), d=rng.choice((256, 1000, 2048, 2056, 4096)), y=rng.choice(("fp32", io)),
                 h=rng.choice(("fp32", io)), io=io, gate=rng.choice(("none", "none", "token", "full")),
                 act=rng.choice(("silu", "sigmoid")), post=rng.random() < 0.5, pre=rng.random() < 0.8,
                 scale=rng.choice((1.0, 0.5)), offset=rng.choice((0.0, 1.0)))


def _lengths(c):
    n, m = [], c["long"]
    for s in range(c["seqs"]):
        n.append(max(1, round(c["q"] * c["spread"] ** (-s / max(m - 1, 1)))) if s < m else 1)
    return n


# ----------------------------------------------------------------- prepare --
def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    io = DTYPES[c["io"]]
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    unif = lambda lo, hi, *s: lo + (hi - lo) * torch.rand(*s, device="cuda", generator=gen)
    if c["op"] in ("gated", "block"):
        n, d = c["tokens"], c["d"]
        st = dict(c=c)
        if c["op"] == "gated":
            h = c["heads"]
            st["o"] = rand(n, h, d).to(io)
            # the gate is a slice of a wider projection
            st["z"] = rand(n, h + 1, d).to(io)[:, :h]
            st["w"] = (rand(d) * 0.2 + (0.0 if c["offset"] else 1.0)).to(io)
            st["out"] = torch.empty(n, h, d, dtype=io, device="cuda")
            if own:
                from expert_cached_decode_gb300 import moe_norm_gated
                st["call"] = moe_norm_gated
            return st
        st["y"] = (rand(n, d) * 0.3).to(DTYPES[c["y"]])
        st["h"] = (rand(n, d) * 2).to(DTYPES[c["h"]])
        w = lambda: (rand(d) * 0.2 + (0.0 if c["offset"] else 1.0)).to(io)
        st["pre_w"], st["post_w"] = w() if c["pre"] else None, w() if c["post"] else None
        st["gate"] = {"none": None, "token": rand(n, 1).to(io), "full": rand(n, d).to(io)}[c["gate"]]
        st["h_out"] = torch.empty_like(st["h"])
        st["x"] = torch.empty(n, d, dtype=io, device="cuda") if c["pre"] else None
        if own:
            from expert_cached_decode_gb300 import moe_norm_block
            st["call"] = moe_norm_block
        return st
    lens = _lengths(c)
    S, T = len(lens), sum(lens)
    wide = 2 * c["hk"] * c["dk"] + c["hv"] * c["dv"]
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    order = torch.randperm(2 * S, device="cuda", generator=gen).to(torch.int32)
    s_in = torch.full((S,), -1, dtype=torch.int32, device="cuda") if c["fresh"] else order[:S].clone()
    s_out = order[S:].clone() if c["keep"] or c["fresh"] else order[:S].clone()
    # what the gates are made of, as models start out: decays of 0.001 to 0.1 a step and head, times 1 to 16
    dt = torch.exp(unif(math.log(1e-3), math.log(0.1), c["hv"]))
    a_log, dt_bias = torch.log(unif(1.0, 16.0, c["hv"])), torch.log(torch.expm1(dt))
    st = dict(c=c, cu=cu, s_in=s_in, s_out=s_out, max_q=max(lens))
    if c["op"] == "prepare":
        st["x"] = rand(T, wide).to(io)
        st["a"], st["b"] = rand(T, c["hv"]).to(io), rand(T, c["hv"]).to(io)
        st["conv_w"] = (rand(wide, c["taps"]) * 0.5).to(io)
        st["a_log"], st["dt_bias"] = a_log, dt_bias
        st["conv"] = rand(2 * S, c["taps"] - 1, wide).to(io)
        st["y"] = torch.empty(T, wide, dtype=io, device="cuda")
        st["g"], st["beta"] = (torch.empty(T, c["hv"], device="cuda") for _ in range(2))
    else:
        x = rand(T, wide)
        x = x * torch.sigmoid(x)
        nq = c["hk"] * c["dk"]
        if not c["normalize"]:
            # a model that norms q and k itself
            qk = x[:, :2 * nq].view(T, 2 * c["hk"], c["dk"])
            x[:, :2 * nq] = (qk * torch.rsqrt(qk.square().sum(-1, keepdim=True) + EPS)).view(T, -1)
        x = x.to(io)
        st["q"], st["k"] = x[:, :nq].view(T, c["hk"], c["dk"]), x[:, nq:2 * nq].view(T, c["hk"], c["dk"])
        st["v"] = x[:, 2 * nq:].view(T, c["hv"], c["dv"])
        st["g"] = -torch.exp(a_log) * torch.log1p(torch.exp(rand(T, c["hv"]) + dt_bias))
        st["beta"] = torch.sigmoid(rand(T, c["hv"]))
        st["state"] = rand(2 * S, c["hv"], c["dk"], c["dv"]) * 0.1
        st["out"] = torch.empty(T, c["hv"], c["dv"], dtype=io, device="cuda")
    if own:
        from expert_cached_decode_gb300 import GatedDelta
        st["op"] = GatedDelta(c["hk"], c["hv"], c["dk"], c["dv"], dtype=io, taps=c["taps"], normalize=c["normalize"], eps=EPS)
    return st


# --------------------------------------------------------------------- run --
def run(st):
    c = st["c"]
    if own:
        if c["op"] == "gated":
            st["call"](st["o"], st["z"], st["w"], st["out"], act=c["act"], gate_first=c["first"], eps=EPS, weight_offset=c["offset"])
            return st["out"]
        if c["op"] == "block":
            st["call"](st["y"], st["h"], st["h_out"], st["x"], pre_w=st["pre_w"], post_w=st["post_w"], gate=st["gate"],
                       act=c["act"], scale=c["scale"], eps=EPS, weight_offset=c["offset"])
            return [st["h_out"], st["x"]]
        if c["op"] == "prepare":
            st["op"].moe_delta_prepare(st["x"], st["conv_w"], None, st["conv"], st["y"], st["a"], st["b"], st["a_log"],
                                       st["dt_bias"], st["g"], st["beta"], st["cu"], st["s_in"], st["s_out"])
            return [st["y"], st["g"], st["beta"], st["conv"]]
        st["op"].moe_delta_forward(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], st["out"], st["cu"],
                                   st["s_in"], st["s_out"], max_q=st["max_q"])
        return [st["out"], st["state"]]
    return {"gated": _plain_gated, "block": _plain_block, "prepare": _plain_prepare, "delta": _plain_delta}[c["op"]](st)


def _act(x, kind):
    return torch.sigmoid(x) if kind == "sigmoid" else x * torch.sigmoid(x)


def _rms(x, w, offset):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (w.float() + offset)


def _plain_gated(st):
    c, o, g = st["c"], st["o"].float(), _act(st["z"].float(), st["c"]["act"])
    st["out"].copy_(_rms(o * g, st["w"], c["offset"]) if c["first"] else _rms(o, st["w"], c["offset"]) * g)
    return st["out"]


def _plain_block(st):
    c, y = st["c"], st["y"].float()
    if st["post_w"] is not None:
        y = _rms(y, st["post_w"], c["offset"])
    if st["gate"] is not None:
        y = y * _act(st["gate"].float(), c["act"])
    h = st["h"].float() + c["scale"] * y
    st["h_out"].copy_(h)
    if st["x"] is not None:
        st["x"].copy_(_rms(h, st["pre_w"], c["offset"]))
    return [st["h_out"], st["x"]]


def _places(st):
    """Sequence of each token, and its place there."""
    cu = st["cu"].long()
    t = torch.arange(st["x" if "x" in st else "q"].shape[0], device=cu.device)
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return t, s, t - cu[s]


def _plain_prepare(st):
    c, taps = st["c"], st["c"]["taps"]
    t, s, place = _places(st)
    old = torch.where((st["s_in"] >= 0)[:, None, None], st["conv"][st["s_in"].clamp(min=0).long()].float(), 0.0)
    x, w = st["x"].float(), st["conv_w"].float()
    y = torch.zeros_like(x)
    for i in range(taps):
        back = taps - 1 - i                          # the input `back` tokens ago: of this call, or kept from before
        past = old[s, (taps - 1 + place - back).clamp(0, taps - 2)]
        y += w[:, i] * torch.where((place >= back)[:, None], x[(t - back).clamp(min=0)], past)
    st["y"].copy_(_act(y, "silu"))
    cu = st["cu"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(taps - 1, device=x.device)
    at = n[:, None] - (taps - 1) + j                 # place of the j-th input that is kept
    rows = torch.arange(len(n), device=x.device)[:, None]
    new = torch.where((at >= 0)[..., None], x[(cu[:-1, None] + at).clamp(min=0)], old[rows, (taps - 1 + at).clamp(0, taps - 2)])
    st["conv"][st["s_out"].long()] = new.to(st["conv"].dtype)
    z = st["a"].float() + st["dt_bias"]
    st["g"].copy_(-torch.exp(st["a_log"]) * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))))
    st["beta"].copy_(torch.sigmoid(st["b"].float()))
    return [st["y"], st["g"], st["beta"], st["conv"]]


def _inverse(a):
    """(1 + a)^-1 for strictly lower triangular a: the inverses of two diagonal blocks give that of both together."""
    n = a.shape[-1]
    inv = torch.eye(n, device=a.device).expand_as(a).clone()
    m = 1
    while m < n:
        b = inv.unflatten(-1, (n // (2 * m), 2 * m)).unflatten(-3, (n // (2 * m), 2 * m))
        e = a.unflatten(-1, (n // (2 * m), 2 * m)).unflatten(-3, (n // (2 * m), 2 * m))
        b, e = (torch.diagonal(v, dim1=-4, dim2=-2).movedim(-1, -3) for v in (b, e))
        b[..., m:, :m] = -(b[..., m:, m:] @ (e[..., m:, :m] @ b[..., :m, :m]))
        m *= 2
    return inv


def _plain_delta(st):
    c = st["c"]
    dev = st["q"].device
    S, hv, rep = c["seqs"], c["hv"], c["hv"] // c["hk"]
    C = 1 << min(6, max(0, (st["max_q"] - 1).bit_length()))
    N = -(-st["max_q"] // C)
    cu = st["cu"].long()
    place = torch.arange(N * C, device=dev)
    real = place < (cu[1:] - cu[:-1])[:, None]                        # [S, N C]
    tok = torch.where(real, cu[:-1, None] + place, 0)

    def chunks(x):                                                    # [T, H, ...] -> [N, S, H, C, ...], zeros behind the end
        x = x.float()[tok] * real.view(S, N * C, *[1] * (x.dim() - 1))
        return x.unflatten(1, (N, C)).movedim(1, 0).movedim(3, 2)

    def unit(x):
        x = x.float()
        return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS) if c["normalize"] else x

    q = chunks(unit(st["q"])).repeat_interleave(rep, 2) * c["dk"] ** -0.5
    k, v = chunks(unit(st["k"])).repeat_interleave(rep, 2), chunks(st["v"])
    beta = chunks(st["beta"])
    G = chunks(st["g"]).double().cumsum(-1)                           # long sums of decays, and their differences
    low = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    D = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    eG, rest = G.exp().float(), (G[..., -1:] - G).exp().float()
    inv = _inverse((beta[..., None] * D * (k @ k.mT)).tril(-1))
    P = D * (q @ k.mT)
    s_in = st["s_in"].long()
    state = torch.where((s_in >= 0).view(S, 1, 1, 1), st["state"][s_in.clamp(min=0)], 0.0)
    out = torch.empty(S, N * C, hv, c["dv"], device=dev)
    for i in range(N):
        z = beta[i][..., None] * (v[i] - eG[i][..., None] * (k[i] @ state))
        u = inv[i] @ z
        o = eG[i][..., None] * (q[i] @ state) + P[i] @ u
        out[:, i * C:(i + 1) * C] = o.movedim(1, 2)
        state = eG[i][..., -1:, None] * state + (rest[i][..., None] * k[i]).mT @ u
    st["out"].copy_(out[real])
    st["state"][st["s_out"].long()] = state
    return [st["out"], st["state"]]


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """The definitions in 64 bits, token by token where they are a recurrence."""
    st = prepare(case, seed)
    c = st["c"]
    f = lambda name: None if st[name] is None else st[name].double()
    sig = lambda x: 1 / (1 + torch.exp(-x))
    gate = lambda x: sig(x) if c["act"] == "sigmoid" else x * sig(x)
    norm = lambda x, w: x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * (c["offset"] + w)
    if c["op"] == "gated":
        return norm(f("o") * gate(f("z")), f("w")) if c["first"] else norm(f("o"), f("w")) * gate(f("z"))
    if c["op"] == "block":
        y = f("y") if st["post_w"] is None else norm(f("y"), f("post_w"))
        h = f("h") + c["scale"] * (y if st["gate"] is None else gate(f("gate")) * y)
        return [h, None if st["x"] is None else norm(h, f("pre_w"))]
    ends = st["cu"].tolist()
    s_in, s_out = st["s_in"].tolist(), st["s_out"].tolist()
    if c["op"] == "prepare":
        x, w, conv = f("x"), f("conv_w"), f("conv")
        y, new = torch.empty_like(x), conv.clone()
        for s in range(c["seqs"]):
            old = conv[s_in[s]] if s_in[s] >= 0 else torch.zeros_like(conv[0])
            both = torch.cat([old, x[ends[s]:ends[s + 1]]])
            n = ends[s + 1] - ends[s]
            r = sum(w[:, i] * both[i:i + n] for i in range(c["taps"]))
            y[ends[s]:ends[s + 1]] = r * sig(r)
            new[s_out[s]] = both[n:]
        g = -torch.exp(f("a_log")) * torch.log1p(torch.exp(f("a") + f("dt_bias")))
        return [y, g, sig(f("b")), new]
    lens = _lengths(c)
    q, k, v, g, beta = f("q"), f("k"), f("v"), f("g"), f("beta")
    if c["normalize"]:
        q, k = (x / (x.pow(2).sum(-1, keepdim=True) + EPS).sqrt() for x in (q, k))
    q, k = (x.repeat_interleave(c["hv"] // c["hk"], 1) for x in (q / math.sqrt(c["dk"]), k))
    pool, out = f("state"), torch.empty_like(v)
    # the sequences longest first, so that those still running are the first ones
    order = sorted(range(len(lens)), key=lambda s: -lens[s])
    S = torch.stack([pool[s_in[s]] if s_in[s] >= 0 else torch.zeros_like(pool[0]) for s in order])
    first = torch.tensor([ends[s] for s in order], device=v.device)
    left = len(order)
    for i in range(max(lens)):
        while lens[order[left - 1]] <= i:
            left -= 1
        t = first[:left] + i
        A = S[:left]
        A *= torch.exp(g[t])[..., None, None]
        kt = k[t]
        u = beta[t][..., None] * (v[t] - (kt[..., None, :] @ A)[..., 0, :])
        A += kt[..., :, None] * u[..., None, :]
        out[t] = (q[t][..., None, :] @ A)[..., 0, :]
    for r, s in enumerate(order):
        pool[s_out[s]] = S[r]
    return [out, pool]


# -------------------------------------------------------------------- work --
def work(case):
    c = case
    e = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "gated":
        n = c["tokens"] * c["heads"] * c["d"]
        return {"bytes": 3 * n * 2 + c["d"] * 2, "flops": 8 * n}
    if c["op"] == "block":
        n = c["tokens"] * c["d"]
        gate = {"none": 0, "token": c["tokens"] * 2, "full": n * 2}[c["gate"]]
        return {"bytes": n * (e[c["y"]] + 2 * e[c["h"]] + 2 * c["pre"]) + gate + 2 * c["d"] * (c["pre"] + c["post"]), "flops": 10 * n}
    lens = _lengths(c)
    T, S = sum(lens), len(lens)
    wide = 2 * c["hk"] * c["dk"] + c["hv"] * c["dv"]
    back = 1 if c["fresh"] else 2                    # states written, and read
    if c["op"] == "prepare":
        return {"bytes": 2 * T * wide * 2 + T * c["hv"] * 12 + back * S * (c["taps"] - 1) * wide * 2 + wide * c["taps"] * 2,
                "flops": T * (wide * (2 * c["taps"] + 4) + 20 * c["hv"])}
    return {"bytes": T * (wide * 2 + c["hv"] * (c["dv"] * 2 + 8)) + back * S * c["hv"] * c["dk"] * c["dv"] * 4,
            "flops": 6 * T * c["hv"] * c["dk"] * c["dv"]}
