"""Linear attention with a decay a head and the step between blocks, in 64 bits and token by token, and
how far the library may be from them: every rounding counted, relative to sums of absolute values."""
import math

import torch

D = 128
U16 = 2.0 ** -8   # half a step of bf16, relative
U32 = 2.0 ** -24  # of fp32
GROUP = 128       # tokens that the library's prefill takes together


def tokens(q, k, v, g, S=None, scale=1.0):
    """One sequence: q, k [n, Hk, D], v [n, H, D], g [n, H], S [H, D, D] or None.  The outputs [n, H, D] and the
    states after 0, 1, .. n tokens, in 64 bits."""
    n, H = v.shape[:2]
    r = H // q.shape[1]
    q, k = (x.double().repeat_interleave(r, 1) for x in (q, k))
    v, a = v.double(), torch.exp(g.double())
    S = torch.zeros(H, D, D, dtype=torch.float64) if S is None else S.double()
    o, states = torch.empty_like(v), [S]
    for t in range(n):
        S = torch.where(a[t, :, None, None] == 0, 0.0, a[t, :, None, None] * S) + k[t, :, :, None] * v[t, :, None, :]
        o[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
        states.append(S)
    return o, states


def stage(o, gate, weight, eps):
    """sigmoid(gate) * weight * o / rms(o)."""
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.double()
    return torch.sigmoid(gate.double()) * w * o / torch.sqrt(o.pow(2).mean(-1, keepdim=True) + eps)


def stage_far(o, far, gate, weight, eps):
    """How far the stage's result may be off when o is off by `far`: by o itself, and by the root mean square, which
    is off by no more than that of `far`; and a few roundings of its own."""
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.double().abs()
    rms = torch.sqrt(o.pow(2).mean(-1, keepdim=True) + eps)
    off = far.pow(2).mean(-1, keepdim=True).sqrt()
    low = torch.clamp(rms - off, min=math.sqrt(eps) if eps else 1e-300)
    part = torch.sigmoid(gate.double()) * w * (far / low + o.abs() * off / (rms * low))
    return part + 64 * U32 * stage(o, gate, weight, eps).abs()


def prefill_far(q, k, v, g, S, scale):
    """(o, final state): how far before o's own rounding.  With absolute values in their places the recurrence gives
    the sums that the errors are relative to.  o: the state in front of a chunk is rounded to bf16 (a half step),
    the chunk's weights to two bf16 parts (a half step of what the first leaves; a part that is zero is exact), a state has its
    own error, sums and decays of 32 bits: a twentieth of a half step more; exponents up to E have lost E 2^-24 twice, in units of ln 2.  States: decayed
    values in three bf16 parts (2^-21 left over at most), 128 products a chunk and one step a chunk in 32 bits, decays within 2^-21."""
    A, states = tokens(q.abs(), k.abs(), v.abs(), g, None if S is None else S.abs(), abs(scale))
    n = v.shape[0]
    deepest = max((float(-g[i:i + GROUP].double().clamp(min=-192 * math.log(2)).sum(0).min()) for i in range(0, n, GROUP)), default=0.0)
    state = 0.0 if S is None and n <= GROUP else 1.0  # none in front of a first chunk
    return A * ((state + 0.05) * U16 + U16 * U16 + 4 * deepest * U32), states[-1] * (2.0 ** -21 + GROUP * 2 * U32 + (n // GROUP + 2) * 2.0 ** -21)


def decode_far(q, k, v, g, S, scale):
    """(o, states after each token): a dot product of 128 terms, a few products, decays within 2 steps: 64 roundings."""
    A, states = tokens(q.abs(), k.abs(), v.abs(), g, S.abs(), abs(scale))
    return 64 * U32 * A, [64 * U32 * s for s in states]


def check(got, want, far, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), finite), f"{what}: finite in other places"
    off = (got - want)[finite].abs() - far[finite] - 1e-37
    assert not bool((off > 0).any()), f"{what}: {int((off > 0).sum())} of {off.numel()} values off, by up to {float(off.max()):.3g}"


def block(x, weight, y=None, post_norm=False, post_weight=None, gate=None, scale=1.0, eps=1e-5):
    """(h, x') and how far each may be off, x' before its rounding."""
    rms = lambda t: torch.sqrt(t.pow(2).mean(-1, keepdim=True) + eps)  # noqa: E731
    x = x.double()
    sums = x.abs()
    if y is not None:
        y = y.double()
        if post_norm:
            y = y / rms(y)
        if post_weight is not None:
            y = y * post_weight.double()
        if gate is not None:
            y = y * torch.sigmoid(gate.double())
        x, sums = x + scale * y, sums + (scale * y).abs()
    far = 2.0 ** -19 * sums  # a norm, a gate and three products in 32 bits: fast exponentials lose 2^-24 of up to 16
    w = torch.ones(x.shape[1], dtype=torch.float64) if weight is None else weight.double()
    h = w * x / rms(x)
    off = far.pow(2).mean(-1, keepdim=True).sqrt() / rms(x)
    return h, x, w.abs() * far / rms(x) + h.abs() * (off + 2.0 ** -19), far
