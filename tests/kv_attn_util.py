"""Plain statements, in 64 bits, of the attention cache's operators, and the error bounds that
their arithmetic allows (independent of the library).

Bounds.  A rounding is off by half a step: bf16 2^-8, f16 2^-11, fp32 2^-24 of the value.
  score x_j = scale q . k_j: 128 fp32 products and sums, the scale's and the exponent's
      roundings: |dx| <= 136 * 2^-24 * scale * sum|q||k_j| + 4 * 2^-24 * (|x_j| + |max x|)
  weight p_j: e^dx, the exponential's 2^-21, and one rounding to the values' type
      (bf16 2^-8; f16 2^-11 and at most 2^-25 of the largest weight)
  sums over n keys: n * 2^-24
  o: the weights' error times sum_j w_j |v_j|, and o's own rounding 2^-8 |o|.
"""
import math

import torch

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
D = 128


def pow2(e):
    return torch.tensor([2.0 ** int(i) for i in e.reshape(-1)], dtype=torch.float64).reshape(e.shape)


def quantise(x):
    """Rows of 128 (any float type) -> (codes' values in 64 bits, scale bytes), element by element
    from the definition: the least whole e in [-40, 40] with max|x| <= 448 * 2^e, then the
    nearest of the e4m3 values, ties to the even code."""
    x = x.double()
    codes = torch.arange(0, 127, dtype=torch.int64)  # the non-negative finite values in order
    ex, man = codes >> 3, (codes & 7).double()
    grid = torch.where(ex == 0, man * 2.0 ** -9, (1 + man / 8) * pow2(ex - 7))
    flat = x.reshape(-1, D)
    out = torch.zeros_like(flat)
    byte = torch.zeros(flat.shape[0], dtype=torch.uint8)
    for i, row in enumerate(flat):
        top = float(row.abs().max())
        if not math.isfinite(top) or top > 448.0 * 2.0 ** 40:
            byte[i] = 255
            continue
        e = -40
        while 448.0 * 2.0 ** e < top:
            e += 1
        y = (row / 2.0 ** e).abs()
        hi = torch.searchsorted(grid, y).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dl, dh = y - grid[lo], grid[hi] - y
        pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        out[i] = torch.where(row < 0, -grid[pick], grid[pick])
        byte[i] = e + 127
    return out.reshape(x.shape), byte.reshape(x.shape[:-1])


def stored(x, fp8):
    """What a cache holds of bf16 rows: (pool rows in the pool's type, scale bytes or None, values in 64 bits)."""
    if not fp8:
        return x.to(torch.bfloat16), None, x.to(torch.bfloat16).double()
    codes, byte = quantise(x)
    size = torch.where(byte == 255, math.nan, pow2(byte.to(torch.int64).clamp(max=254) - 127))
    return codes.to(torch.float8_e4m3fn), byte, codes * size[..., None]


def visible(n, total, window, sink):
    p = torch.arange(total - n, total)[:, None]
    j = torch.arange(total)
    see = j <= p
    if window:
        see &= (p - j < window) | (j < sink)
    return see


def attention(q, k, v, see, scale, fp8):
    """One sequence: q [n, H, D], k, v [total, Hkv, D] in 64 bits, see [n, total].  Returns o, lse and their bounds."""
    n, H, _ = q.shape
    total, Hkv, _ = k.shape
    G = H // Hkv
    o, lse = torch.zeros(n, H, D, dtype=torch.float64), torch.full((n, H), -math.inf, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    if total == 0:
        return o, lse, bo, bl
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[:, h // G], v[:, h // G]
        some = see.any(1)
        x = torch.where(see, qh @ torch.where(torch.isfinite(kh), kh, 0.0).T * scale, -math.inf)
        mass = torch.where(see, qh.abs() @ torch.where(torch.isfinite(kh), kh, 0.0).abs().T * abs(scale), 0.0)
        y = torch.logsumexp(x, 1)
        w = torch.where(some[:, None], torch.exp(x - torch.where(some, y, 0.0)[:, None]), 0.0)
        clean = torch.where(torch.isfinite(vh), vh, 0.0)
        oh, spread = w @ clean, w @ clean.abs()
        top = torch.where(see, x.abs(), 0.0).amax(1)
        dx = 136 * F32 * mass.amax(1) + 8 * F32 * top
        # f16 weights are relative to the largest weight times value scale: its 2^-25 counts once a key
        wt = F16 + 2.0 ** -25 * total if fp8 else BF16
        rel = 2 * dx + 2.0 ** -20 + 2 * total * F32 + wt
        largest = torch.where(see[:, :, None], clean.abs(), 0.0).amax(1) if fp8 else torch.zeros(n, D, dtype=torch.float64)
        bo[:, h] = BF16 * oh.abs() + 1.01 * rel[:, None] * spread + (2.0 ** -24 * total * w.amax(1)[:, None] * largest if fp8 else 0)
        bl[:, h] = dx + 2.0 ** -20 + total * F32 + 4 * F32 * torch.where(some, y, 0.0).abs()
        o[:, h] = oh
        lse[:, h] = y
        # rows that see a key row or value row with a NaN or an infinity
        broken = ~torch.isfinite(kh).all(1) | ~torch.isfinite(vh).all(1)
        o[(see & broken).any(1), h] = math.nan
    return o, lse, bo, bl


class Cache:
    """A paged cache on the device, filled row by row from the sequences' keys and values.

    ``layout``: "heads" [page][head][token], "tokens" [page][token][head], or "pair" k and v of a
    page in one allocation.  Unused slots hold NaN (and NaN codes, scale bytes 255 or 0)."""

    def __init__(self, lens, Hkv, page, fp8, gen, layout="heads", spare=2, values=None, max_pages=None, device="cuda"):
        self.fp8, self.page, self.Hkv = fp8, page, Hkv
        n_of = [(t + page - 1) // page for t in lens]
        n_pages = sum(n_of) + spare
        perm = torch.randperm(n_pages, generator=gen)
        width = max(max(n_of), 1) if max_pages is None else max_pages
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        shape = (n_pages, Hkv, page, D)
        pool = {}
        self.value = {"k": [], "v": []}
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        scale = {}
        for n in ("k", "v"):
            pool[n] = torch.full(shape, math.nan).to(kind)
            scale[n] = torch.full(shape[:3], 255, dtype=torch.uint8)
            scale[n][::2] = 0
        at = 0
        for i, t in enumerate(lens):
            pages = perm[at:at + n_of[i]]
            at += n_of[i]
            table[i, :n_of[i]] = pages.to(torch.int32)
            for n in ("k", "v"):
                x = torch.randn(t, Hkv, D, generator=gen) * torch.exp2(torch.randn(t, Hkv, 1, generator=gen))
                x = x.to(torch.bfloat16)
                if values is not None:
                    x = values(n, i, x)
                rows, byte, val = stored(x, fp8)
                self.value[n].append(val)
                for j in range(n_of[i]):
                    m = min(page, t - j * page)
                    pool[n].view(torch.uint8 if fp8 else torch.int16)[pages[j], :, :m] = (
                        rows[j * page:j * page + m].transpose(0, 1).contiguous().view(torch.uint8 if fp8 else torch.int16))
                    if fp8:
                        scale[n][pages[j], :, :m] = byte[j * page:j * page + m].T
        self.table = table.to(device)
        raw = torch.uint8 if fp8 else torch.int16
        if layout == "heads":
            self.k, self.v = pool["k"].to(device), pool["v"].to(device)
        elif layout == "tokens":
            self.k, self.v = (pool[n].view(raw).transpose(1, 2).contiguous().to(device).view(kind).transpose(1, 2) for n in ("k", "v"))
        else:
            both = torch.stack([pool["k"].view(raw), pool["v"].view(raw)], 1).to(device).view(kind)
            self.k, self.v = both[:, 0], both[:, 1]
        self.scales = dict(k_scale=scale["k"].to(device), v_scale=scale["v"].to(device)) if fp8 else {}
        self.args = (self.k, self.v, self.table)


def check(o, lse, ref):
    """Every element of o and lse within its bound, non-finite exactly where the reference says."""
    ro, rl, bo, bl = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    nan = torch.isnan(ro).any(-1)
    assert torch.equal(~torch.isfinite(o).all(-1), nan), "rows non-finite where they should not be, or the other way round"
    err = (o - ro).abs()[~nan]
    assert (err <= bo[~nan]).all(), f"o off by {float((err / bo[~nan].clamp(min=1e-300)).max()):.3g} times its bound"
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty)
    assert (o[empty] == 0).all()
    ok = ~nan & ~empty
    err = (lse - rl).abs()[ok]
    assert (err <= bl[ok]).all(), f"lse off by {float((err / bl[ok]).max()):.3g} times its bound"
