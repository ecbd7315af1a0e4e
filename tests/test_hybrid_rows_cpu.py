"""The hybrid example leaves the rows that it is given as they are (no GPU needed: the library's calls are stand-ins)."""
import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from kimi_delta_attention_prefill_gb300.hybrid import HybridStack


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("step", [False, True])
def test_the_residual_stream_is_the_stack_s_own(monkeypatch, dtype, step):
    def block_norm(x, weight, y=None, x_out=None, **kw):
        if y is not None:
            x = torch.add(x, y.float(), out=x_out)
        return x.to(torch.bfloat16), x

    monkeypatch.setattr(kda, "block_norm", block_norm)
    monkeypatch.setattr(kda, "lin_prefill", lambda q, k, v, *a, **kw: (v.contiguous(), None))
    monkeypatch.setattr(kda, "lin_decode", lambda q, k, v, *a, **kw: v.float())
    stack = HybridStack(heads=2, kv_heads=1, width=64, n_seq=3, max_tokens=64, kinds=["decay", "decay"], post_norm=True, device="cpu")
    x = torch.randn(3, 2, 64).to(dtype)
    given = x.clone()
    stack.decode(x) if step else stack.prompt(x.view(6, 64), torch.tensor([0, 2, 4, 6], dtype=torch.int32))
    assert torch.equal(x, given)
