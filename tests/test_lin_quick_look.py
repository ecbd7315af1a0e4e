"""The quick look that linear attention's calls and the step between blocks take at their arguments first, on
tensors that say they are on device 0 (no GPU needed): sound ones pass it, and with others the error names the
argument, whatever its rank or type."""
import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from test_streams import BF, F32, I32, Device, fakes  # noqa: F401 (fixture)


class OnZero(Device):
    def get_device(self):
        return 0


class Stream:
    cuda_stream = 7777
    device = torch.device("cuda", 0)


def dev(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnZero)


def prefill(**kw):
    a = dict(q=dev(5, 2, 128), k=dev(5, 2, 128), v=dev(5, 4, 128), g=dev(5, 4, dtype=F32), cu_seqlens=dev(2, dtype=I32),
             gate=dev(5, 4, 128), norm_weight=dev(128, dtype=F32))
    return kda.lin_prefill(**{**a, **kw}, stream=Stream())


def decode(**kw):
    a = dict(q=dev(2, 3, 2, 128), k=dev(2, 3, 2, 128), v=dev(2, 3, 4, 128), g=dev(2, 3, 4, dtype=F32), gate=dev(2, 3, 4, 128),
             norm_weight=dev(128, dtype=F32), S_state=dev(2, 4, 128, 128, dtype=F32))
    return kda.lin_decode(**{**a, **kw}, stream=Stream())


def norm(**kw):
    a = dict(x=dev(5, 64), weight=dev(64, dtype=F32), y=dev(5, 64), gate=dev(5, 64), post_weight=dev(64, dtype=F32))
    return kda.block_norm(**{**a, **kw}, stream=Stream())


@pytest.mark.parametrize("call,kw", [
    (prefill, {}), (prefill, dict(gate=None, norm_weight=None)), (prefill, dict(norm_weight=None)), (prefill, dict(g=dev(4, dtype=F32))),
    (prefill, dict(v=dev(5, 9, 128)[:, 1:5], gate=dev(7, 6, 128)[1:6, :4])), (decode, {}), (decode, dict(g=dev(4, dtype=F32))),
    (decode, dict(gate=None, norm_weight=None, n_commit=dev(2, dtype=I32))), (norm, {}), (norm, dict(x=dev(5, 64, dtype=F32))),
    (norm, dict(y=None, gate=None, post_weight=None)), (norm, dict(x=dev(5, 80)[:, :64], y=dev(5, 72)[:, 8:]))])
def test_sound_tensors_pass(fakes, monkeypatch, call, kw):  # noqa: F811
    def slow(*a):
        raise AssertionError("the quick look did not take them")

    monkeypatch.setattr(kda, "_say_lin_rows", slow)
    monkeypatch.setattr(kda, "_wide_rows", slow)
    call(**kw)


@pytest.mark.parametrize("call,name,bad", [
    (prefill, "gate", dev(5, 512)), (prefill, "gate", dev(1, 5, 4, 128)), (prefill, "gate", dev(5)), (prefill, "gate", dev(5, 2, 128)),
    (prefill, "gate", dev(5, 4, 256)[..., ::2]), (prefill, "norm_weight", dev(4, 128, dtype=F32)), (prefill, "q", dev(5, 256)),
    (prefill, "k", dev(5, 256)), (prefill, "k", dev(1, 5, 2, 128)), (prefill, "v", dev(5, 512)), (prefill, "v", dev(1, 5, 4, 128)),
    (prefill, "g", dev(5, 4, 1, dtype=F32)), (prefill, "g", dev(dtype=F32)), (prefill, "cu_seqlens", dev(dtype=I32)),
    (prefill, "S_in", dev(1, 4, 16384, dtype=F32)), (prefill, "o", dev(5, 512)), (prefill, "S_out", dev(4, 128, 128, dtype=F32)),
    (decode, "gate", dev(2, 3, 512)), (decode, "gate", dev(6, 4, 128)), (decode, "gate", dev(2, 512)), (decode, "gate", dev(2, 3, 2, 128)),
    (decode, "norm_weight", dev(4, 128, dtype=F32)), (decode, "q", dev(6, 2, 128)), (decode, "k", dev(6, 2, 128)),
    (decode, "v", dev(6, 4, 128)), (decode, "g", dev(6, 4, dtype=F32)), (decode, "g", dev(2, 3, 4, 1, dtype=F32)),
    (decode, "S_state", dev(4, 128, 128, dtype=F32)), (decode, "n_commit", dev(2, 1, dtype=I32)), (decode, "o", dev(6, 4, 128, dtype=F32)),
    (norm, "x", dev(5, 8, 8)), (norm, "x", dev(64)), (norm, "y", dev(5, 8, 8)), (norm, "y", dev(64)), (norm, "gate", dev(64)),
    (norm, "gate", dev(5, 8, 8)), (norm, "weight", dev(1, 64, dtype=F32)), (norm, "post_weight", dev(8, 8, dtype=F32)),
    (norm, "h", dev(64)), (norm, "x_out", dev(1, 5, 64)),
])
def test_ranks_and_shapes(fakes, call, name, bad):  # noqa: F811
    """A projection's rows before they are split into heads, a dimension too many, and the like."""
    with pytest.raises(ValueError, match=name):
        call(**{name: bad})


@pytest.mark.parametrize("call,name", [
    (prefill, "q"), (prefill, "k"), (prefill, "v"), (prefill, "g"), (prefill, "cu_seqlens"), (prefill, "gate"), (prefill, "norm_weight"),
    (prefill, "S_in"), (prefill, "o"), (prefill, "S_out"), (prefill, "workspace"), (prefill, "dev_status"),
    (decode, "q"), (decode, "k"), (decode, "v"), (decode, "g"), (decode, "gate"), (decode, "norm_weight"), (decode, "S_state"),
    (decode, "n_commit"), (decode, "o"), (decode, "dev_status"),
    (norm, "x"), (norm, "weight"), (norm, "y"), (norm, "gate"), (norm, "post_weight"), (norm, "h"), (norm, "x_out"),
])
@pytest.mark.parametrize("bad", [[1.0], 1, "rows"])
def test_what_is_no_tensor(fakes, call, name, bad):  # noqa: F811
    with pytest.raises((TypeError, ValueError), match=name):
        call(**{name: bad})
