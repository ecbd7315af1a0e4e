"""Arguments that the binding must not pass on to the library as they are (no GPU needed): the library
and the tensors' device are test_streams.py's stand-ins."""
import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from test_streams import F32, I32, Stream, dev, fakes  # noqa: F401 (fixture)


def with_workspace():
    rows, gates = [dev(5, 2, 128) for _ in range(3)], [dev(5, 2, 128, dtype=F32), dev(5, 2, dtype=F32)]
    step = [t.unsqueeze(0)[:, :4] for t in rows + gates]
    cu, table, one = dev(2, dtype=I32), dev(1, 4, dtype=I32), dev(1, dtype=I32)
    pool, state = dev(8, 2, 16, 128), dev(2, 128, 128, dtype=F32)
    return {
        "prefill": lambda w: kda.prefill(*rows, *gates, cu, workspace=w, stream=Stream()),
        "prefill_paged": lambda w: kda.prefill_paged(*rows, *gates, cu, state, workspace=w, stream=Stream()),
        "decode_paged": lambda w: kda.decode_paged(*step, state, dev(2, dtype=I32), workspace=w, stream=Stream()),
        "attn_prefill_paged": lambda w: kda.attn_prefill_paged(rows[0], pool, pool, table, cu, one, workspace=w, stream=Stream()),
        "attn_decode_paged": lambda w: kda.attn_decode_paged(step[0], pool, pool, table, one, workspace=w, stream=Stream()),
    }


@pytest.mark.parametrize("name", sorted(with_workspace()))
def test_workspace_on_the_host_or_in_pieces_is_refused(fakes, name):  # noqa: F811
    """The kernels would write through a host address, or past the end of a strided tensor."""
    call = with_workspace()[name]
    call(dev(512, dtype=torch.uint8))
    call(dev(64, dtype=torch.float64))  # any type, as bytes
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        call(torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(dev(1024, dtype=torch.uint8)[::2])
    with pytest.raises(TypeError, match="workspace"):
        call(bytearray(512))


@pytest.mark.parametrize("name", ["attn_prefill_paged", "attn_decode_paged"])
def test_window_and_first_tokens_past_32_bits(fakes, monkeypatch, name):  # noqa: F811
    """A window wider than any sequence is no window, not what is left of its low 32 bits."""
    got = []
    entry = getattr(kda.library(), "kda_" + name)
    lib = kda.library()
    monkeypatch.setattr(type(lib), "kda_" + name, lambda self, *a: (got.append(a), entry(*a))[1], raising=False)
    rows, table, one = dev(4, 2, 128), dev(1, 4, dtype=I32), dev(1, dtype=I32)
    pool = dev(8, 2, 16, 128)
    q, more = (rows, (dev(2, dtype=I32), one)) if "prefill" in name else (rows[None], (one,))
    at = 12 if "prefill" in name else 11  # window, n_sink
    for value, want in ((2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 40, 2 ** 31 - 1), (-1, -1), (-2 ** 32 + 5, -1), (7, 7)):
        getattr(kda, name)(q, pool, pool, table, *more, window=value, n_sink=value, stream=Stream())
        assert got[-1][at:at + 2] == (want, want)
