"""Linear attention with a decay a head, and the norms around a block: cases, inputs, plain forms.

A hybrid stack may hold layers whose memory is a 128 x 128 state a head that only decays and adds,

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,      o_t = scale * S_t^T q_t,

with one log-decay g <= 0 a (token, head), or one a head.  Groups of heads may share their q and k.
Three operators serve such a layer:

  prefill  packed sequences from their entry states: every token's output, and the final states
  decode   1 to 4 tokens of each sequence; the state after the accepted ones replaces the old one
  norm     the step between two blocks over the residual stream x: with a block's output y,
           x' = x + scale * sigmoid(gate) * weight * y / rms(y),  and the next block's input
           h = weight' * x' / rms(x');  all parts but the last are optional

prefill and decode also run with the layer's output stage in them, sigmoid(gate) * weight * o / rms(o)
over a head's channels.  128 channels a head throughout.
"""
import math
import random

import torch

own = False

D = 128
EPS = 1e-5
DEV = "cuda"


def listed():
    def lin(name, op, **kw):
        d = dict(name=name, op=op, heads=96, qk_heads=96, seqs=1, new=1, ragged=0, fixed=False, entry=False, gated=False, scaled=False)
        d.update(kw)
        return d

    def norm(name, **kw):
        d = dict(name=name, op="norm", rows=1, width=512, wide=False, block=True, post=False, gated=False, scale=1.0)
        d.update(kw)
        return d

    return [
        # short prompts of three conversations that go on: latency
        lin("prefill short", "prefill", heads=16, qk_heads=4, seqs=3, new=97, ragged=1, entry=True),
        # the model-width prompt: 8192 tokens, 96 heads
        lin("prefill prompt", "prefill", new=8192),
        # a batch of ragged prompts, q and k shared by groups of four, with the output stage
        lin("prefill batch", "prefill", heads=64, qk_heads=16, seqs=12, new=4001, ragged=2, entry=True, gated=True, scaled=True),
        # one very long prompt on few heads, a decay a head: the sequence has to be split over the machine
        lin("prefill long", "prefill", heads=8, qk_heads=8, new=262144, fixed=True),
        # one conversation's next token: latency
        lin("decode one", "decode", heads=32, qk_heads=8),
        # a full decode batch at model width: bandwidth
        lin("decode batch", "decode", seqs=256),
        # a verify step of 4 tokens, some accepted, with the output stage
        lin("verify batch", "decode", heads=64, qk_heads=16, seqs=61, new=4, ragged=3, gated=True, scaled=True),
        # a small stack's step between blocks: latency
        norm("norm step", rows=3, width=512, post=True),
        # a decode batch at model width (96 heads of 128), all parts
        norm("norm decode", rows=256, width=12288, post=True, gated=True, scale=0.5),
        # the model-width prompt, all parts: bandwidth
        norm("norm prompt", rows=8192, width=12288, post=True, gated=True, scale=0.5),
        # a residual stream of 32 bits, an odd number of rows, a width that is no power of two, no gate
        norm("norm wide", rows=30001, width=1928, wide=True, post=True),
        # the norm before the first block
        norm("norm first", rows=4001, width=5128, block=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "norm", "norm"])
        yes = lambda p: rng.random() < p  # noqa: E731
        if op == "norm":
            block = yes(0.8)
            c = dict(op=op, rows=_log(rng, 1, 30000), width=8 * _log(rng, 16, 2048), wide=yes(0.3), block=block,
                     post=block and yes(0.6), gated=block and yes(0.4), scale=rng.choice([1.0, 0.5, 0.1767]) if block else 1.0)
            if c["rows"] * c["width"] > 100e6:
                continue
            return c
        shared = rng.choice([1, 2, 4, 8, 16, 32])
        c = dict(op=op, heads=shared * rng.choice([1, 1, 2, 3, 4, 6]), qk_heads=shared, seqs=1, new=1, ragged=rng.randrange(1, 1000),
                 fixed=yes(0.3), entry=yes(0.5), gated=yes(0.4), scaled=yes(0.5))
        if op == "decode":
            c.update(seqs=_log(rng, 1, 256), new=rng.randint(1, 4), entry=False)
            if c["seqs"] * c["heads"] <= 256 * 96:
                return c
        else:
            c.update(seqs=_log(rng, 1, 48), new=_log(rng, 1, 100000))
            chunks = -(-c["new"] // CHUNK)
            units = c["seqs"] * c["heads"]
            if units * chunks <= 16384 and units * chunks * chunks <= 34e6:
                return c


def _lengths(case):
    """New tokens of each sequence: the first has the most, the others spread below it."""
    r = random.Random(case["ragged"])
    out = []
    for i in range(case["seqs"]):
        n = case["new"] if i == 0 or not case["ragged"] else 1 + int(case["new"] * r.random())
        if case["ragged"] and i % 5 == 4:
            n = 1
        out.append(min(n, case["new"]))
    return out


def _commits(case):
    r = random.Random(case["ragged"] + 1)
    return [r.randint(0, case["new"]) if case["ragged"] else case["new"] for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        res = 4 if case["wide"] else 2
        per = res + 2 + ((2 + res) if case["block"] else 0) + (2 if case["gated"] else 0)
        return {"bytes": n * per + 4 * case["width"] * (2 if case["post"] else 1),
                "flops": n * (4 + (8 if case["block"] else 0))}
    h, hk = case["heads"], case["qk_heads"]
    state = 4 * D * D * h
    if case["op"] == "decode":
        tokens = case["seqs"] * case["new"]
        row = 2 * D * (2 * hk + h + (h if case["gated"] else 0)) + 4 * D * h
        states = case["seqs"] + sum(1 for n in _commits(case) if n)
    else:
        tokens = sum(_lengths(case))
        row = 2 * D * (2 * hk + 2 * h + (h if case["gated"] else 0))
        states = case["seqs"] * (2 if case["entry"] else 1)
    row += 0 if case["fixed"] else 4 * h
    return {"bytes": tokens * row + states * state, "flops": 4 * D * D * h * tokens}


# ------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def rand(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)

    s = {"case": case}
    if case["op"] == "norm":
        shape = (case["rows"], case["width"])
        s["x"] = rand(*shape, dtype=torch.float32 if case["wide"] else torch.bfloat16)
        s["weight"] = 1.0 + 0.1 * rand(case["width"])
        s["y"] = rand(*shape, dtype=torch.bfloat16) if case["block"] else None
        s["post_weight"] = 1.0 + 0.1 * rand(case["width"]) if case["post"] else None
        s["gate"] = rand(*shape, dtype=torch.bfloat16) if case["gated"] else None
        return s
    h, hk, step = case["heads"], case["qk_heads"], case["op"] == "decode"
    lens = [case["new"]] * case["seqs"] if step else _lengths(case)
    lead = (case["seqs"], case["new"]) if step else (sum(lens),)

    def unit():
        x = rand(*lead, hk, D, dtype=torch.bfloat16)
        return x.div_(x.float().square().sum(-1, keepdim=True).sqrt().to(torch.bfloat16))

    s["q"], s["k"], s["v"] = unit(), unit(), rand(*lead, h, D, dtype=torch.bfloat16)
    if case["fixed"]:  # memories of a few tokens up to a few hundred
        s["g"] = -torch.exp2(-8.0 * torch.arange(1, h + 1, device=DEV) / h)
    else:  # by token; heads of short and of long memory
        s["g"] = -5.0 * torch.sigmoid(rand(*lead, h) - 4.0 + torch.linspace(-3.0, 2.0, h, device=DEV))
    s["gate"] = rand(*lead, h, D, dtype=torch.bfloat16) if case["gated"] else None
    s["norm_weight"] = 1.0 + 0.1 * rand(D) if case["gated"] else None
    s["scale"] = D ** -0.5 if case["scaled"] else 1.0
    state = (case["seqs"], h, D, D)
    if step:
        s["state"] = rand(*state).mul_(0.1)
        s["n_commit"] = torch.tensor(_commits(case), dtype=torch.int32, device=DEV)
    else:
        s["state"] = rand(*state).mul_(0.1) if case["entry"] else None
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
        s["cu_seqlens"] = cu.to(torch.int32).to(DEV)
        s["longest"] = max(lens)
    return s


# ---------------------------------------------------------------------------------- plain form
def _rms(x):
    return torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if c["block"]:
        y = s["y"].float()
        if c["post"]:
            y = y / _rms(y) * s["post_weight"]
        if c["gated"]:
            y = y * torch.sigmoid(s["gate"].float())
        x = x + c["scale"] * y
    h = (x / _rms(x) * s["weight"]).to(torch.bfloat16)
    return {"h": h, "x": x.to(s["x"].dtype)} if c["block"] else {"h": h}


def _stage(s, o, dtype):
    """Scale, and the output stage where there is one, rounded once."""
    o = o * s["scale"]
    if s["gate"] is not None:
        o = o / _rms(o) * s["norm_weight"] * torch.sigmoid(s["gate"].float())
    return o.to(dtype)


CHUNK = 128  # tokens that the plain form takes together


def _plain_prefill(s):
    """The sequences padded to N x C chunks.  Within a chunk ((q k^T) * decays) v; a chunk's entry state is
    the sum of the earlier chunks' k^T v, each times the decays in between."""
    c = s["case"]
    N, H, Hk, L = c["seqs"], c["heads"], c["qk_heads"], CHUNK
    C = -(-s["longest"] // L)
    cu = s["cu_seqlens"].long()
    T = s["v"].shape[0]
    i = torch.arange(C * L, device=DEV)
    live = i < (cu[1:] - cu[:-1])[:, None]                     # [N, C L]
    at = (cu[:-1, None] + i).clamp(max=T - 1)

    def padded(x):                                             # [N, heads, C, L, D]
        x = torch.where(live[..., None, None], x[at].float(), 0.0)
        return x.view(N, C, L, -1, D).permute(0, 3, 1, 2, 4)

    q, k, v = (padded(s[n]) for n in ("q", "k", "v"))
    q, k = (x.repeat_interleave(H // Hk, 1) for x in (q, k))
    g = s["g"].double().expand(T, H)[at].masked_fill(~live[..., None], 0.0)
    g = g.view(N, C, L, H).permute(0, 3, 1, 2)
    G = g.cumsum(-1)                                           # [N, H, C, L], inclusive, in the chunk
    last = G[..., -1:]
    kv = torch.matmul((k * torch.exp(last - G)[..., None].float()).transpose(-1, -2), v)
    # weights of chunk b's k^T v and of S_in in the state before chunk a (a = C: at the end)
    B = torch.cat([torch.zeros_like(last[:, :, :1, 0]), last[..., 0].cumsum(-1)], -1)  # [N, H, C + 1]
    w = B[..., :, None] - B[..., None, 1:]
    w.masked_fill_(torch.arange(C + 1, device=DEV)[:, None] <= torch.arange(C, device=DEV), -math.inf)
    E = torch.matmul(torch.exp(w).float(), kv.reshape(N, H, C, D * D))
    if s["state"] is not None:
        E += torch.exp(B).float()[..., None] * s["state"].reshape(N, H, 1, D * D)
    E = E.view(N, H, C + 1, D, D)
    x = G[..., :, None] - G[..., None, :]
    x.masked_fill_(torch.ones(L, L, dtype=torch.bool, device=DEV).triu(1), -math.inf)
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * torch.exp(x).float(), v)
    o += torch.exp(G).float()[..., None] * torch.matmul(q, E[:, :, :-1])
    o = o.permute(0, 2, 3, 1, 4).reshape(N * C * L, H, D)[live.reshape(-1)]
    return {"o": _stage(s, o, torch.bfloat16), "state": E[:, :, -1].contiguous()}


def _plain_decode(s):
    c = s["case"]
    n, r = c["new"], c["heads"] // c["qk_heads"]
    S = s["state"]
    q, k = (s[x].float().repeat_interleave(r, 2) for x in ("q", "k"))
    v = s["v"].float()
    G = s["g"].double().expand(c["seqs"], n, c["heads"]).cumsum(1)  # [B, n, H]
    x = G[:, :, None] - G[:, None]                                  # [B, t, i, H]
    x = x.masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)[..., None], -math.inf)
    a = torch.exp(x).float() * (q[:, :, None] * k[:, None]).sum(-1)
    o = torch.exp(G).float()[..., None] * torch.matmul(q.transpose(1, 2), S).transpose(1, 2)
    o = o + (a[..., None] * v[:, None]).sum(2)
    # the state after n_commit tokens: none of them leaves it as it was
    m = s["n_commit"].long()
    Gm = torch.where(m[:, None] > 0, G.gather(1, (m - 1).clamp(min=0)[:, None, None].expand(-1, 1, c["heads"]))[:, 0], 0.0)
    wt = torch.where((torch.arange(n, device=DEV) < m[:, None])[..., None], Gm[:, None] - G, -math.inf)
    add = torch.matmul((k * torch.exp(wt).float()[..., None]).permute(0, 2, 3, 1), v.transpose(1, 2))
    S.mul_(torch.exp(Gm).float()[..., None, None]).add_(add)
    return {"o": _stage(s, o, torch.float32), "state": S}


def run(state):
    s = state
    c = s["case"]
    if own:
        import kimi_delta_attention_prefill_gb300 as kda

        if c["op"] == "norm":
            if not c["block"]:
                return {"h": kda.block_norm(s["x"], s["weight"], eps=EPS)[0]}
            h, x = kda.block_norm(s["x"], s["weight"], s["y"], post_norm=c["post"], post_weight=s["post_weight"],
                                  gate=s["gate"], scale=c["scale"], eps=EPS)
            return {"h": h, "x": x}
        stage = dict(scale=s["scale"], gate=s["gate"], norm_weight=s["norm_weight"], eps=EPS)
        if c["op"] == "prefill":
            o, S = kda.lin_prefill(s["q"], s["k"], s["v"], s["g"], s["cu_seqlens"], S_in=s["state"], **stage)
            return {"o": o, "state": S}
        o = kda.lin_decode(s["q"], s["k"], s["v"], s["g"], s["state"], n_commit=s["n_commit"], **stage)
        return {"o": o, "state": s["state"]}
    return {"norm": _plain_norm, "prefill": _plain_prefill, "decode": _plain_decode}[c["op"]](s)


# --------------------------------------------------------------------------------------- exact
def _exact_norm(s):
    c = s["case"]
    out = {"h": torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)}
    if c["block"]:
        out["x"] = torch.empty_like(out["h"])
    for i in range(0, c["rows"], 1024):
        r = slice(i, i + 1024)
        x = s["x"][r].double()
        if c["block"]:
            y = s["y"][r].double()
            if c["post"]:
                y *= s["post_weight"].double() * (y.pow(2).sum(1, keepdim=True) / c["width"] + EPS).rsqrt()
            if c["gated"]:
                y /= 1 + torch.exp(-s["gate"][r].double())
            x += c["scale"] * y
            out["x"][r] = x
        out["h"][r] = x * (x.pow(2).sum(1, keepdim=True) / c["width"] + EPS).rsqrt() * s["weight"].double()
    return out


def _exact_rows(s, S, lo, hi, seq):
    """Tokens lo .. hi (rows of one sequence, few) from the states S [H, D, D] in 64 bits, token by token of
    their cumulative decays: outputs [n, H, D], and the states after each of them by a function."""
    c = s["case"]
    pick = (lambda x: x[seq, lo:hi]) if c["op"] == "decode" else (lambda x: x[lo:hi])
    r = c["heads"] // c["qk_heads"]
    q, k, v = (pick(s[n]).double().transpose(0, 1) for n in ("q", "k", "v"))   # [heads, n, D]
    q, k = q.repeat_interleave(r, 0), k.repeat_interleave(r, 0)
    n = hi - lo
    g = (s["g"].double()[None].expand(n, -1) if c["fixed"] else pick(s["g"]).double()).T.contiguous()
    A = g.cumsum(1)
    decay = torch.exp(torch.where(torch.ones(n, n, device=DEV).tril() > 0, A[:, :, None] - A[:, None, :], -math.inf))
    o = torch.bmm(torch.bmm(q, k.transpose(1, 2)) * decay, v) + torch.exp(A)[..., None] * torch.bmm(q, S)
    o = o.transpose(0, 1) * s["scale"]
    if s["gate"] is not None:
        o = o * (o.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * s["norm_weight"].double()
        o = o / (1 + torch.exp(-pick(s["gate"]).double()))

    def after(m):  # m tokens
        if m == 0:
            return S
        w = torch.exp(A[:, m - 1:m] - A[:, :m])
        return torch.exp(A[:, m - 1])[:, None, None] * S + torch.bmm((k[:, :m] * w[..., None]).transpose(1, 2), v[:, :m])

    return o, after


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    h = case["heads"]
    o = torch.empty(s["v"].shape, dtype=torch.float64, device=DEV)
    states = torch.empty((case["seqs"], h, D, D), dtype=torch.float64, device=DEV)
    if case["op"] == "decode":
        for i, m in enumerate(_commits(case)):
            o[i], after = _exact_rows(s, s["state"][i].double(), 0, case["new"], i)
            states[i] = after(m)
        return {"o": o, "state": states}
    at = 0
    for i, n in enumerate(_lengths(case)):
        S = torch.zeros((h, D, D), dtype=torch.float64, device=DEV) if s["state"] is None else s["state"][i].double()
        for lo in range(at, at + n, 64):
            hi = min(lo + 64, at + n)
            o[lo:hi], after = _exact_rows(s, S, lo, hi, i)
            S = after(hi - lo)
        states[i] = S
        at += n
    return {"o": o, "state": states}
