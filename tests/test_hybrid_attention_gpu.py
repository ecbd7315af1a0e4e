"""The attention layers of the hybrid example, call by call, against the 64-bit statement over what
their cache holds."""
import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from kimi_delta_attention_prefill_gb300.hybrid import HybridStack
from kv_attn_util import D, attention, check, visible

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_tokens,kernel", [(512, 0), (1 << 17, 1)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (100, 4)])
def test_attention_layers(monkeypatch, max_tokens, kernel, fp8, window, n_sink):
    """A prompt in two chunks, a verify step and a single token, through either chunk kernel."""
    calls = []

    def held(k_pool, v_pool, table, lens, scales):
        cu = torch.tensor([0] + lens, dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)
        start = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        return [t.cpu().double().split(lens) for t in kda.kv_read(k_pool, v_pool, table, cu, start, sum(lens), **scales)]

    def compare(q, new, o, lse, k_pool, v_pool, table, kv_len, kw):
        lens = kv_len.tolist()
        k, v = held(k_pool, v_pool, table, lens, {n: kw[n] for n in ("k_scale", "v_scale") if n in kw})
        parts = [attention(x.cpu(), k[i], v[i], visible(new[i], lens[i], kw["window"], kw["n_sink"]), D ** -0.5, fp8)
                 for i, x in enumerate(q.split(new)) if new[i]]
        check(o, lse, [torch.cat(x) for x in zip(*parts)])

    prefill, decode = kda.attn_prefill_paged, kda.attn_decode_paged

    def attn_prefill_paged(q, k_pool, v_pool, table, cu, kv_len, **kw):
        o, lse = prefill(q, k_pool, v_pool, table, cu, kv_len, return_lse=True, **kw)
        calls.append(kda.debug_attention_kernel(table.shape[0], q.shape[0], q.shape[1], k_pool.shape[1], table.shape[1] * k_pool.shape[2]))
        compare(q, cu.diff().tolist(), o, lse, k_pool, v_pool, table, kv_len, kw)
        return o

    def attn_decode_paged(q, k_pool, v_pool, table, kv_len, **kw):
        o, lse = decode(q, k_pool, v_pool, table, kv_len, return_lse=True, **kw)
        calls.append("decode")
        compare(q.flatten(0, 1), [q.shape[1]] * q.shape[0], o.flatten(0, 1), lse.flatten(0, 1), k_pool, v_pool, table, kv_len, kw)
        return o

    monkeypatch.setattr(kda, "attn_prefill_paged", attn_prefill_paged)
    monkeypatch.setattr(kda, "attn_decode_paged", attn_decode_paged)
    stack = HybridStack(n_layers=3, period=2, n_seq=3, max_tokens=max_tokens, fp8=fp8, window=window, n_sink=n_sink, page_size=32)
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    cu = lambda new: torch.tensor([0] + new, dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)
    for new in ([200, 41, 1], [130, 60, 7]):
        stack.prompt(rows(sum(new), 512), cu(new))
    for n_tok in (3, 1):
        stack.decode(rows(3, n_tok, 512))
    torch.cuda.synchronize()
    assert int(stack.status) == 0
    assert stack.length.tolist() == [334, 105, 12]
    assert calls == [kernel, kernel, "decode", "decode"]
