"""The attention cache's operators, as a serving loop calls them: cases, inputs, plain forms.

A hybrid stack runs delta-rule layers next to layers of softmax attention, and the latter keep
a cache of keys and values in pages.  Four operators serve it:

  append   new tokens' keys and values into their pages, as bf16 or quantised to e4m3 with one
           power-of-two scale per (token, head)
  read     a range of cached tokens back as packed bf16 rows (hand-over of a prefix)
  chunk    attention of a chunk of new tokens of each sequence over its paged cache
  decode   the same for 1 to 4 tokens of each sequence

chunk and decode also run with a sliding window and a few first tokens that stay visible.
Everything is 128 channels a head.  Page p of head h holds page_size consecutive tokens:
pools are [n_pages, kv_heads, page_size, 128], page tables [sequences, pages] int32 (-1: none).
"""
import math
import random

import torch

own = False

D = 128
E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = -40, 40  # exponents that a scale may have; its byte is the exponent + 127, 255 = NaN row
DEV = "cuda"


def listed():
    def c(name, op, **kw):
        d = dict(name=name, op=op, kv="bf16", heads=96, kv_heads=8, page=64, seqs=1, new=1, past=0, ragged=0, window=0, sink=0)
        d.update(kw)
        return d

    return [
        # a decode step of 256 sequences puts one token each into an e4m3 cache: latency
        c("append step", "append", kv="fp8", seqs=256, new=1, past=500, ragged=1),
        # the chunks of five prompts, odd lengths, e4m3
        c("append prompts", "append", kv="fp8", seqs=5, new=4001, past=777, ragged=2),
        # a whole prefix imported into a bf16 cache: bandwidth
        c("append import", "append", seqs=16, new=16384, past=100, ragged=3, page=128),
        # a short cached prefix handed on
        c("read prefix", "read", kv="fp8", seqs=3, new=2500, ragged=4, page=16),
        # a batch's cache moved to another worker: bandwidth
        c("read batch", "read", kv="fp8", seqs=64, new=8192, ragged=5),
        # a few tokens of three conversations over short pasts: latency
        c("chunk small", "chunk", heads=16, kv_heads=2, seqs=3, new=33, past=1500, ragged=6, page=16),
        # the model-width prompt (8192 tokens, 96 heads) from an empty cache
        c("chunk prompt", "chunk", new=8192),
        # a later chunk of a long prompt over an e4m3 cache
        c("chunk long", "chunk", kv="fp8", new=2048, past=30001),
        # ragged prompts under a window with first tokens kept
        c("chunk window", "chunk", seqs=4, new=4096, past=2000, ragged=7, window=1024, sink=4, page=32),
        # one conversation's next token: latency
        c("decode one", "decode", past=5000),
        # a full decode batch over an e4m3 cache: bandwidth
        c("decode batch", "decode", kv="fp8", seqs=256, past=8191, ragged=8),
        # a verify step of 4 tokens under a window with first tokens kept
        c("verify window", "decode", heads=64, seqs=64, new=4, past=30000, ragged=9, window=4096, sink=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "read", "chunk", "chunk", "chunk", "decode", "decode", "decode"])
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
        c = dict(op=op, kv=rng.choice(["bf16", "fp8"]), heads=kv_heads * group, kv_heads=kv_heads,
                 page=rng.choice([16, 32, 64, 128]), seqs=1, new=1, past=0, ragged=rng.randrange(1, 1000), window=0, sink=0)
        if op in ("append", "read"):
            c.update(seqs=_log(rng, 1, 256), new=_log(rng, 1, 16384), past=_log(rng, 1, 8192))
        elif op == "chunk":
            c.update(seqs=_log(rng, 1, 16), new=_log(rng, 1, 8192), past=_log(rng, 1, 30000) - 1)
        else:
            c.update(seqs=_log(rng, 1, 256), new=rng.randint(1, 4), past=_log(rng, 1, 30000))
        if op in ("chunk", "decode") and rng.random() < 0.35:
            c.update(window=_log(rng, 16, 8192), sink=rng.choice([0, 1, 4, 64]))
        rows = _lengths(c)
        tokens, held = sum(n for n, _ in rows), sum(t for _, t in rows)
        w = work(c)
        scores = c["seqs"] * c["heads"] * max(n for n, _ in rows) * max(t for _, t in rows)
        if w["flops"] <= 2.5e12 and w["bytes"] <= 1.5e9 and scores <= 3e9 and max(tokens, held) * kv_heads <= 4.5e6:
            return c


def _lengths(case):
    """(new tokens, tokens in the cache after them) of each sequence.  With ragged = 0 all are the
    same; otherwise the first has the most and the others spread below it."""
    r = random.Random(case["ragged"])
    out = []
    for i in range(case["seqs"]):
        full = not case["ragged"] or i == 0
        fixed = full or case["op"] == "decode"
        n = case["new"] if fixed else 1 + int(case["new"] * r.random())
        p = case["past"] if full else int(case["past"] * r.random())
        if not fixed and i % 5 == 4:
            n = 1
        out.append((min(n, case["new"]), p + min(n, case["new"])))
    return out


def _seen(case, n, total):
    """(query, key) pairs that a sequence's mask leaves, and the keys that any query sees."""
    w, s = case["window"], case["sink"]
    if not w:
        return n * total - n * (n - 1) // 2, total
    pairs = 0
    first = total - n
    for p in range(first, total):
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(s, lo)
    lo = max(0, first - w + 1)
    return pairs, total - lo + min(s, lo)


def work(case):
    rows = _lengths(case)
    held = 1 if case["kv"] == "fp8" else 2
    scale = 1 if case["kv"] == "fp8" else 0
    hk, h = case["kv_heads"], case["heads"]
    new = sum(n for n, _ in rows)
    if case["op"] in ("append", "read"):
        return {"bytes": 2 * new * hk * (2 * D + held * D + scale), "flops": 2 * new * hk * D}
    pairs = keys = 0
    for n, t in rows:
        a, b = _seen(case, n, t)
        pairs, keys = pairs + a, keys + b
    return {"bytes": 2 * keys * hk * (held * D + scale) + new * h * (4 * D + 4), "flops": 4 * D * h * pairs}


# ------------------------------------------------------------------------------------- inputs
def _pow2(e):
    """2^e of whole e in [-127, 127], in 64 bits and exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise(x):
    """e4m3 codes and scale bytes of rows of 128: the smallest power of two 2^e (e within
    [SCALE_MIN, SCALE_MAX]) with max|x| <= 448 * 2^e, codes the nearest e4m3 to x / 2^e (ties to
    even).  A row with a NaN, an infinity or a value above 448 * 2^SCALE_MAX holds zeros and byte 255."""
    x = x.float()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top > 0, e, SCALE_MIN).clamp(min=SCALE_MIN)
    bad = ~(top <= E4M3_MAX * 2.0 ** SCALE_MAX)
    e = torch.where(bad, 0, e)
    codes = (x * _pow2(-e)[..., None].float()).masked_fill(bad[..., None], 0.0).to(torch.float8_e4m3fn)
    return codes, torch.where(bad, 255, e + 127).to(torch.uint8)


def _rows(gen, shape):
    """Keys or values as a model makes them: unit scale, tokens of different size, a few large channels."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    size = torch.exp2(torch.randn(shape[:-1] + (1,), generator=gen, device=DEV) * 0.5).to(torch.bfloat16)
    channel = torch.ones(shape[-1], device=DEV, dtype=torch.bfloat16)
    channel[::37] = 4.0
    return x.mul_(size).mul_(channel)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rows = _lengths(case)
    P, hk, fp8 = case["page"], case["kv_heads"], case["kv"] == "fp8"
    s = {"case": case, "new": [n for n, _ in rows]}
    news = torch.tensor([n for n, _ in rows], dtype=torch.int64)
    totals = torch.tensor([t for _, t in rows], dtype=torch.int64)
    n_of = (totals + P - 1) // P
    n_pages, width = int(n_of.sum()) + 3, int(n_of.max())
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    first = (n_of.cumsum(0) - n_of).to(DEV)
    col = torch.arange(width, device=DEV)
    table = perm[(first[:, None] + col).clamp(max=n_pages - 1)]
    s["page_table"] = torch.where(col < n_of.to(DEV)[:, None], table, -1).contiguous()
    s["cu_seqlens"] = torch.cat([torch.zeros(1, dtype=torch.int64), news.cumsum(0)]).to(torch.int32).to(DEV)
    s["start"] = (totals - news).to(torch.int32).to(DEV)
    s["kv_len"] = totals.to(torch.int32).to(DEV)
    T = int(news.sum())
    s["T"], s["longest"], s["most"] = T, int(news.max()), int(totals.max())
    pool = (n_pages, hk, P, D)
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    if case["op"] == "append":
        s["k"], s["v"] = _rows(gen, (T, hk, D)), _rows(gen, (T, hk, D))
        s["k_pool"], s["v_pool"] = (torch.zeros(pool, dtype=torch.uint8 if fp8 else kind, device=DEV).view(kind) for _ in range(2))
        s["k_scale"], s["v_scale"] = (torch.full(pool[:3], 127, dtype=torch.uint8, device=DEV) if fp8 else None for _ in range(2))
        return s
    for n in ("k", "v"):
        x = _rows(gen, pool)
        if fp8:
            codes, scale = torch.empty(pool, dtype=kind, device=DEV), torch.empty(pool[:3], dtype=torch.uint8, device=DEV)
            step = max(1, (1 << 28) // (hk * P * D))
            for i in range(0, n_pages, step):
                codes[i:i + step], scale[i:i + step] = _quantise(x[i:i + step])
            s[n + "_pool"], s[n + "_scale"] = codes, scale
        else:
            s[n + "_pool"], s[n + "_scale"] = x, None
    shape = (case["seqs"], case["new"], case["heads"], D) if case["op"] == "decode" else (T, case["heads"], D)
    if case["op"] != "read":
        s["q"] = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------------- plain form
def _positions(s):
    """Sequence and position in the cache of each packed token."""
    t = torch.arange(s["T"], device=DEV)
    cu = s["cu_seqlens"].long()
    seq = torch.bucketize(t, cu[1:], right=True)
    return seq, s["start"].long()[seq] + t - cu[seq]


def _plain_append(s):
    P = s["case"]["page"]
    seq, pos = _positions(s)
    page, slot = s["page_table"][seq, pos // P].long(), pos % P
    for n in ("k", "v"):
        if s[n + "_scale"] is None:
            s[n + "_pool"][page, :, slot] = s[n]
        else:
            codes, scale = _quantise(s[n])
            s[n + "_pool"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            s[n + "_scale"][page, :, slot] = scale


def _value(codes, scale):
    """What codes and scale bytes stand for, in 32 bits."""
    size = torch.where(scale == 255, math.nan, _pow2(scale.clamp(max=254).int() - 127)).float()
    return codes.float().mul_(size[..., None])


def _held(s, n, page, slot=None):
    """Rows of a pool as 32-bit values: whole pages, or one slot of each."""
    at = (page,) if slot is None else (page, slice(None), slot)
    x = s[n + "_pool"]
    if s[n + "_scale"] is None:
        return x[at].float()
    return _value(x.view(torch.uint8)[at].view(torch.float8_e4m3fn), s[n + "_scale"][at])


def _plain_read(s):
    P = s["case"]["page"]
    seq, pos = _positions(s)
    page, slot = s["page_table"][seq, pos // P].long(), pos % P
    return tuple(_held(s, n, page, slot).to(torch.bfloat16) for n in ("k", "v"))


def _plain_attention(s):
    """softmax(q k^T / sqrt(128)) v over the padded batch, and the log of each row's sum."""
    c = s["case"]
    N, hk, G = c["seqs"], c["kv_heads"], c["heads"] // c["kv_heads"]
    n, L = s["longest"], s["page_table"].shape[1] * c["page"]
    page = s["page_table"].clamp(min=0).long()
    k, v = (_held(s, x, page).permute(0, 2, 1, 3, 4).reshape(N, hk, L, D) for x in ("k", "v"))
    total = s["kv_len"].long()
    if c["op"] == "decode":
        q = s["q"]
        pos = total[:, None] - n + torch.arange(n, device=DEV)
    else:
        cu = s["cu_seqlens"].long()
        i = torch.arange(n, device=DEV)
        q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)]
        pos = (total - (cu[1:] - cu[:-1]))[:, None] + i
    q = q.float().view(N, n, hk, G, D).permute(0, 2, 1, 3, 4).reshape(N, hk, n * G, D)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    j = torch.arange(L, device=DEV)
    see = (j <= pos[..., None]) & (j < total[:, None, None])
    if c["window"]:
        see &= (j > pos[..., None] - c["window"]) | (j < c["sink"])
    x.view(N, hk, n, G, L).masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.sub_(top).exp_()
    total_p = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v).div_(torch.where(total_p > 0, total_p, 1.0))
    lse = (top + total_p.log())[..., 0]
    o = o.view(N, hk, n, G, D).permute(0, 2, 1, 3, 4).reshape(N, n, hk * G, D)
    lse = lse.view(N, hk, n, G).permute(0, 2, 1, 3).reshape(N, n, hk * G)
    if c["op"] != "decode":
        seq, pos = _positions(s)
        i = pos - s["start"].long()[seq]
        o, lse = o[seq, i], lse[seq, i]
    return o.to(torch.bfloat16), lse.contiguous()


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import kimi_delta_attention_prefill_gb300 as kda

        pool = (s["k_pool"], s["v_pool"], s["page_table"])
        scale = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
        seen = dict(window=s["case"]["window"], n_sink=s["case"]["sink"], return_lse=True)
        if op == "append":
            kda.kv_append(s["k"], s["v"], *pool, s["cu_seqlens"], s["start"], **scale)
        elif op == "read":
            k, v = kda.kv_read(*pool, s["cu_seqlens"], s["start"], s["T"], **scale)
        elif op == "chunk":
            o, lse = kda.attn_prefill_paged(s["q"], *pool, s["cu_seqlens"], s["kv_len"], **scale, **seen)
        else:
            o, lse = kda.attn_decode_paged(s["q"], *pool, s["kv_len"], **scale, **seen)
    elif op == "append":
        _plain_append(s)
    elif op == "read":
        k, v = _plain_read(s)
    else:
        o, lse = _plain_attention(s)
    if op == "append":
        return {n: s[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale")}
    return {"k": k, "v": v} if op == "read" else {"o": o, "lse": lse}


# --------------------------------------------------------------------------------------- exact
def _grid(x):
    """x (64 bits) in rows of 128 as the quantised cache holds it: (codes' values, exponent)."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(SCALE_MIN, SCALE_MAX)
    e = torch.where(E4M3_MAX * _pow2(e - 1) >= top, e - 1, e)  # the logarithm's own rounding
    e = torch.where(E4M3_MAX * _pow2(e) < top, e + 1, e).clamp(SCALE_MIN, SCALE_MAX)
    y = x / _pow2(e)
    step = _pow2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(y / step) * step, e


def _table_rows(s, i, lo, hi):
    """(pages, slots) of tokens lo .. hi of sequence i."""
    j = torch.arange(lo, hi, device=DEV)
    return s["page_table"][i].long()[j // s["case"]["page"]], j % s["case"]["page"]


def _value64(s, n, page, h, slot):
    if s[n + "_scale"] is None:
        return s[n + "_pool"][page, h, slot].double()
    codes = s[n + "_pool"].view(torch.uint8)[page, h, slot].view(torch.float8_e4m3fn).double()
    return codes * _pow2(s[n + "_scale"][page, h, slot].int() - 127)[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    rows = _lengths(case)
    hk, G = case["kv_heads"], case["heads"] // case["kv_heads"]
    if case["op"] == "append":
        out = {"k_scale": None, "v_scale": None}
        for n in ("k", "v"):
            out[n + "_pool"] = torch.zeros(s[n + "_pool"].shape, dtype=torch.float64, device=DEV)
            at = 0
            for i, (new, total) in enumerate(rows):
                page, slot = _table_rows(s, i, total - new, total)
                x = s[n][at:at + new].double()
                out[n + "_pool"][page, :, slot] = x if s[n + "_scale"] is None else _grid(x)[0]
                at += new
        return out
    if case["op"] == "read":
        out = {n: torch.empty((s["T"], hk, D), dtype=torch.float64, device=DEV) for n in ("k", "v")}
        at = 0
        for i, (new, total) in enumerate(rows):
            page, slot = _table_rows(s, i, total - new, total)
            for h in range(hk):
                for n in ("k", "v"):
                    out[n][at:at + new, h] = _value64(s, n, page, h, slot)
            at += new
        return out
    q = s["q"].reshape(-1, case["heads"], D)
    o = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
    at = 0
    for i, (new, total) in enumerate(rows):
        page, slot = _table_rows(s, i, 0, total)
        p = torch.arange(total - new, total, device=DEV)[:, None]
        j = torch.arange(total, device=DEV)
        hidden = j > p
        if case["window"]:
            hidden |= (p - j >= case["window"]) & (j >= case["sink"])
        for h in range(hk):
            k, v = (_value64(s, n, page, h, slot) for n in ("k", "v"))
            for g in range(h * G, (h + 1) * G):
                x = q[at:at + new, g].double() @ k.T / math.sqrt(D)
                x[hidden] = -math.inf
                y = torch.logsumexp(x, 1)
                lse[at:at + new, g] = y
                o[at:at + new, g] = torch.exp(x - y[:, None]) @ v
        at += new
    return {"o": o.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}
