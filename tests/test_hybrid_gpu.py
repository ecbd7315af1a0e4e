"""The hybrid example: delta-rule and attention layers served together."""
import pytest
import torch

from kimi_delta_attention_prefill_gb300.hybrid import HybridStack, main

pytestmark = pytest.mark.gpu

# Each layer's output is within 1e-2 of its maximum (the library's bar for o) in either run, the
# residual stream passes a layer's error on, and two runs of four layers are compared.
TOL = 2 * 4 * 1e-2


def cu(new):
    return torch.tensor([0] + list(new), dtype=torch.int32, device="cuda").cumsum(0, dtype=torch.int32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (100, 4)])
def test_chunks_and_single_tokens_continue_a_prompt(fp8, window, n_sink):
    """A prompt in chunks, then a verify step of 3 tokens and a single token, gives what the
    whole prompt gives at once."""
    lens = [300, 45, 5]
    kw = dict(n_seq=3, max_tokens=512, fp8=fp8, window=window, n_sink=n_sink, page_size=32)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = [torch.randn(n, 512, generator=g, device="cuda", dtype=torch.bfloat16) for n in lens]
    whole = HybridStack(**kw)
    want = whole.prompt(torch.cat(x), cu(lens)).split(lens)
    parts = HybridStack(**kw)
    got = [[], [], []]
    cuts = [[0, 128, 190, 296], [0, 1, 20, 41], [0, 0, 1, 1]]
    for c in range(3):
        new = [cuts[i][c + 1] - cuts[i][c] for i in range(3)]
        y = parts.prompt(torch.cat([x[i][cuts[i][c]:cuts[i][c + 1]] for i in range(3)]), cu(new)).split(new)
        for i in range(3):
            got[i].append(y[i])
    for n in (3, 1):
        at = [sum(t.shape[0] for t in got[i]) for i in range(3)]
        y = parts.decode(torch.stack([x[i][at[i]:at[i] + n] for i in range(3)]))
        for i in range(3):
            got[i].append(y[i])
    torch.cuda.synchronize()
    assert int(whole.status) == 0 and int(parts.status) == 0
    assert parts.length.tolist() == lens
    for i in range(3):
        a, b = torch.cat(got[i]).float(), want[i].float()
        assert a.shape == b.shape
        assert float((a - b).abs().max() / b.abs().max()) <= TOL


def test_example_runs(capsys):
    main()
    assert "lengths [303, 80, 4]" in capsys.readouterr().out
