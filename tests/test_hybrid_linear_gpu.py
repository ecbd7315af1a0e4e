"""The hybrid example's layers with a decay a head and the steps between its blocks, call by call against the
64-bit statements, and whole runs against one another."""
import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from kimi_delta_attention_prefill_gb300.hybrid import HybridStack
from lin_util import U16, U32, block, check, decode_far, prefill_far, stage, stage_far, tokens

pytestmark = pytest.mark.gpu

KINDS = ["decay", "attention", "decay", "decay"]


def cu(new):
    return torch.tensor([0] + list(new), dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)


def rows(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def test_each_call(monkeypatch):
    """A prompt in two chunks, a verify step that keeps some of its tokens, a single token."""
    calls = []
    prefill, decode, norm = kda.lin_prefill, kda.lin_decode, kda.block_norm

    def one(q, k, v, g, S, gate, weight):
        g = g.expand(v.shape[0], -1) if g.dim() == 1 else g
        return tuple(t.cpu() for t in (q, k, v, g, S, gate, weight))

    def lin_prefill(q, k, v, g, cu_seqlens, S_in, S_out, gate, norm_weight, dev_status):
        before = S_in.clone()
        o, S = prefill(q, k, v, g, cu_seqlens, S_in=S_in, S_out=S_out, gate=gate, norm_weight=norm_weight, dev_status=dev_status)
        at = cu_seqlens.tolist()
        for i in range(len(at) - 1):
            r = slice(at[i], at[i + 1])
            q1, k1, v1, g1, S0, gate1, w = one(q[r], k[r], v[r], g if g.dim() == 1 else g[r], before[i], gate[r], norm_weight)
            want, states = tokens(q1, k1, v1, g1, S0)
            far, s_far = prefill_far(q1, k1, v1, g1, S0, 1.0)
            far, want = stage_far(want, far, gate1, w, 1e-5), stage(want, gate1, w, 1e-5)
            check(o[r], want, far + U16 * (want.abs() + far), "o")
            check(S[i], states[-1], s_far, "state")
        calls.append("prefill")
        return o, S

    def lin_decode(q, k, v, g, S_state, n_commit, gate, norm_weight, dev_status):
        before, n_tok = S_state.clone(), q.shape[1]
        o = decode(q, k, v, g, S_state, n_commit=n_commit, gate=gate, norm_weight=norm_weight, dev_status=dev_status)
        for i in range(q.shape[0]):
            q1, k1, v1, g1, S0, gate1, w = one(q[i], k[i], v[i], g if g.dim() == 1 else g[i], before[i], gate[i], norm_weight)
            want, states = tokens(q1, k1, v1, g1, S0)
            far, s_far = decode_far(q1, k1, v1, g1, S0, 1.0)
            check(o[i], stage(want, gate1, w, 1e-5), stage_far(want, far, gate1, w, 1e-5), "o")
            n = n_tok if n_commit is None else int(n_commit[i])
            check(S_state[i], states[n], s_far[n], "state")
        calls.append("decode")
        return o

    def block_norm(x, weight, y=None, x_out=None, **kw):
        a = dict(x=x, weight=weight, y=y, **kw)
        a = {n: t.cpu().clone() if isinstance(t, torch.Tensor) else t for n, t in a.items()}
        h, x1 = norm(x, weight, y, x_out=x_out, **kw)
        want_h, want_x, far_h, far_x = block(**a)
        check(h, want_h, far_h + U16 * (want_h.abs() + far_h), "h")
        check(x1, want_x, far_x + U32 * (want_x.abs() + far_x), "x")
        calls.append("norm")
        return h, x1

    for name, f in (("lin_prefill", lin_prefill), ("lin_decode", lin_decode), ("block_norm", block_norm)):
        monkeypatch.setattr(kda, name, f)
    stack = HybridStack(heads=4, kv_heads=2, kinds=KINDS, n_seq=3, max_tokens=512, post_norm=True, block_scale=0.5)
    for c, new in enumerate(([200, 41, 1], [130, 0, 7])):
        stack.prompt(rows(c, sum(new), 512), cu(new))
    keep = torch.tensor([3, 0, 1], dtype=torch.int32, device="cuda")
    stack.decode(rows(7, 3, 4, 512), n_commit=keep)
    stack.decode(rows(8, 3, 1, 512))
    torch.cuda.synchronize()
    assert int(stack.status) == 0 and stack.length.tolist() == [334, 42, 10]
    layers = lambda kind: ["norm", kind, "norm", "norm", kind, "norm", kind, "norm"]  # noqa: E731 (the second is attention)
    assert calls == 2 * layers("prefill") + 2 * layers("decode")


# Each layer's output is within 1e-2 of its maximum in either run, the residual stream passes a layer's
# error on, and two runs of four layers are compared.
TOL = 2 * 4 * 1e-2


@pytest.mark.parametrize("post_norm", [False, True])
def test_chunks_and_refused_tokens_continue_a_prompt(post_norm):
    """A prompt in chunks, a verify step whose last tokens are refused, then the right ones: what the whole prompt
    gives at once."""
    lens = [300, 45, 5]
    kw = dict(kinds=KINDS, n_seq=3, max_tokens=512, page_size=32, post_norm=post_norm, block_scale=0.5)
    x = [rows(10 + i, n, 512) for i, n in enumerate(lens)]
    whole = HybridStack(**kw)
    want = whole.prompt(torch.cat(x), cu(lens)).split(lens)
    parts = HybridStack(**kw)
    got, at = [[], [], []], [0, 0, 0]
    for new in ([128, 1, 0], [160, 37, 0], [7, 2, 0]):
        y = parts.prompt(torch.cat([x[i][at[i]:at[i] + new[i]] for i in range(3)]), cu(new)).split(new)
        for i in range(3):
            got[i].append(y[i])
            at[i] += new[i]
    # four drafted tokens, the last three of the first and the last one of the second wrong
    right = [1, 3, 4]
    draft = torch.stack([torch.cat([x[i][at[i]:at[i] + right[i]], rows(20 + i, 4 - right[i], 512)]) for i in range(3)])
    y = parts.decode(draft, n_commit=torch.tensor(right, dtype=torch.int32, device="cuda"))
    for i in range(3):
        got[i].append(y[i, :right[i]])
        at[i] += right[i]
    new = [lens[i] - at[i] for i in range(3)]
    y = parts.prompt(torch.cat([x[i][at[i]:] for i in range(3)]), cu(new)).split(new)
    torch.cuda.synchronize()
    assert int(whole.status) == 0 and int(parts.status) == 0 and parts.length.tolist() == lens
    for i in range(3):
        a, b = torch.cat(got[i] + [y[i]]).float(), want[i].float()
        assert a.shape == b.shape
        assert float((a - b).abs().max() / b.abs().max()) <= TOL


def test_refusals():
    with pytest.raises(ValueError, match="delta, decay or attention"):
        HybridStack(kinds=["rnn"])
    stack = HybridStack(n_seq=1, max_tokens=64)
    with pytest.raises(ValueError, match="keep every token"):
        stack.decode(rows(0, 1, 2, 512), n_commit=torch.ones(1, dtype=torch.int32, device="cuda"))
