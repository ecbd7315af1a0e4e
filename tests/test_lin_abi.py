"""Linear attention's entry points and the step between blocks reject bad arguments on the host, before any
CUDA call, and the binding rejects bad tensors (no GPU needed)."""
import ctypes

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from kimi_delta_attention_prefill_gb300 import build
from test_streams import BF, F32, I32, NOTES, Stream, dev, fakes  # noqa: F401 (fixture)

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5
HAS_GPU = torch.cuda.is_available()
P = ctypes.c_void_p
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.library()


def i64(*s):
    return (ctypes.c_int64 * len(s))(*s)


def _prefill(lib, q=0x1000, qs=(256, 128), k=0x2000, ks=(256, 128), v=0x3000, vs=(512, 128), g=0x4000, gs=(4, 1), scale=1.0,
             gate=0, gates=(512, 128), weight=0, eps=1e-5, S_in=0, cu=0x5000, n_seq=1, T=5, o=0x6000, S_out=0x7000, Hk=2, H=4,
             d=128, segments=0, ws=0x100000, ws_bytes=1 << 40, status=0):
    return lib.kda_lin_prefill(P(q), i64(*qs), P(k), i64(*ks), P(v), i64(*vs), P(g), i64(*gs), scale, P(gate), i64(*gates),
                               P(weight), eps, P(S_in), P(cu), n_seq, T, P(o), P(S_out), Hk, H, d, segments, P(ws), ws_bytes,
                               P(status), None)


def _decode(lib, q=0x1000, qs=(256, 256, 128), k=0x2000, ks=(256, 256, 128), v=0x3000, vs=(512, 512, 128), g=0x4000,
            gs=(4, 4, 1), scale=1.0, gate=0, gates=(512, 512, 128), weight=0, eps=1e-5, S=0x10000, commit=0, o=0x6000, B=2,
            n_tok=1, Hk=2, H=4, d=128, status=0):
    return lib.kda_lin_decode(P(q), i64(*qs), P(k), i64(*ks), P(v), i64(*vs), P(g), i64(*gs), scale, P(gate), i64(*gates),
                              P(weight), eps, P(S), P(commit), P(o), B, n_tok, Hk, H, d, P(status), None)


@pytest.mark.parametrize("call", [_prefill, _decode])
def test_what_both_refuse(lib, call):
    lead = (256,) if call is _prefill else (256, 256)
    assert call(lib, d=64) == UNSUPPORTED
    assert call(lib, H=0) == INVALID
    assert call(lib, Hk=0) == INVALID
    assert call(lib, H=4, Hk=3) == INVALID
    assert call(lib, H=65536, Hk=1) == UNSUPPORTED
    for name in ("q", "k", "v", "g", "o"):
        assert call(lib, **{name: 0}) == INVALID
    for name in ("q", "k", "v", "o", "gate", "weight"):
        assert call(lib, **{"gate": 0x8000, name: 0x1008}) == ALIGNMENT
    assert call(lib, g=0x4002) == ALIGNMENT
    assert call(lib, status=0x4002) == ALIGNMENT
    for bad in (124, 0, -128, 1 << 40):
        assert call(lib, qs=lead + (bad,)) == ALIGNMENT
        assert call(lib, ks=(bad,) + lead) == ALIGNMENT
        assert call(lib, vs=lead + (bad,)) == ALIGNMENT
        assert call(lib, gate=0x8000, gates=lead + (bad,)) == ALIGNMENT
    assert call(lib, gs=(-1,) * (len(lead) + 1)) == INVALID
    assert call(lib, scale=NAN) == INVALID
    assert call(lib, scale=INF) == INVALID
    for eps in (-1e-5, NAN, INF):
        assert call(lib, gate=0x8000, eps=eps) == INVALID


def test_prefill_refusals(lib):
    assert _prefill(lib, n_seq=-1) == INVALID
    assert _prefill(lib, T=-1) == INVALID
    assert _prefill(lib, T=1 << 31) == INVALID
    assert _prefill(lib, n_seq=0, T=5) == INVALID
    assert _prefill(lib, segments=-1) == INVALID
    assert _prefill(lib, cu=0) == INVALID
    assert _prefill(lib, cu=0x5002) == ALIGNMENT
    assert _prefill(lib, S_in=0x5008) == ALIGNMENT
    assert _prefill(lib, S_out=0x5008) == ALIGNMENT
    assert _prefill(lib, ws=0x100080) == ALIGNMENT
    planned = dict(n_seq=60, T=500)  # more heads of sequences than SMs
    need = lib.kda_lin_prefill_workspace_size(60, 4, 128, 500, 0)
    assert need > 0
    assert _prefill(lib, ws=0, **planned) == WORKSPACE
    assert _prefill(lib, ws_bytes=need - 1, **planned) == WORKSPACE
    assert lib.kda_lin_prefill_workspace_size(1, 4, 128, 5, 0) == 0
    assert _prefill(lib, n_seq=0, T=0, q=0, k=0, v=0, g=0, o=0, cu=0) == OK
    if not HAS_GPU:
        assert _prefill(lib) in (CUDA, UNSUPPORTED)
        assert _prefill(lib, ws=0, ws_bytes=0) in (CUDA, UNSUPPORTED)
        assert _prefill(lib, ws_bytes=need, **planned) in (CUDA, UNSUPPORTED)


def test_decode_refusals(lib):
    assert _decode(lib, n_tok=0) == UNSUPPORTED
    assert _decode(lib, n_tok=5) == UNSUPPORTED
    assert _decode(lib, B=-1) == INVALID
    assert _decode(lib, S=0) == INVALID
    assert _decode(lib, S=0x10008) == ALIGNMENT
    assert _decode(lib, commit=0x4002) == ALIGNMENT
    assert _decode(lib, B=0, q=0, k=0, v=0, g=0, S=0, o=0) == OK
    if not HAS_GPU:
        assert _decode(lib) in (CUDA, UNSUPPORTED)


def test_prefill_workspace_size(lib):
    size = lambda *a: int(lib.kda_lin_prefill_workspace_size(*a))  # noqa: E731
    assert size(1, 4, 64, 5, 0) == size(-1, 4, 128, 5, 0) == size(1, 0, 128, 5, 0) == size(1, 4, 128, -1, 0) == size(1, 4, 128, 5, -1) == 0
    assert size(1, 96, 128, 8192, 0) == size(3, 16, 128, 291, 0) == size(1, 8, 128, 900, 1) == 0  # a block each, no split
    assert 0 < size(2, 96, 128, 8192, 0) < 1 << 20                # more than the SMs: a plan
    assert size(1, 8, 128, 1 << 20, 0) < 32 << 20                 # at most a state for each SM
    assert size(4, 8, 128, 4096, 3) <= size(4, 8, 128, 4096, 8)


def _norm(lib, x=0x1000, dtype=0, xs=64, weight=0x2000, y=0x3000, ys=64, post=1, pw=0x4000, gate=0x5000, gs=64, scale=1.0,
          eps=1e-5, h=0x6000, x_out=0x7000, rows=3, width=64):
    return lib.kda_block_norm(P(x), dtype, xs, P(weight), P(y), ys, post, P(pw), P(gate), gs, scale, eps, P(h), P(x_out), rows,
                              width, None)


def test_norm_refusals(lib):
    assert _norm(lib, dtype=2) == UNSUPPORTED
    for width in (4, 63, 32776):
        assert _norm(lib, width=width) == UNSUPPORTED
    assert _norm(lib, width=0) == INVALID
    assert _norm(lib, rows=-1) == INVALID
    for bad in (NAN, INF):
        assert _norm(lib, scale=bad) == INVALID
        assert _norm(lib, eps=bad) == INVALID
    assert _norm(lib, eps=-1.0) == INVALID
    assert _norm(lib, x=0) == INVALID
    assert _norm(lib, h=0, x_out=0) == INVALID
    assert _norm(lib, y=0) == INVALID                                        # its parts without it
    assert _norm(lib, y=0, post=0, pw=0, gate=0) == INVALID                  # nor a residual sum
    for name in ("x", "weight", "y", "pw", "gate", "h", "x_out"):
        assert _norm(lib, **{name: 0x1008}) == ALIGNMENT
    for name in ("xs", "ys", "gs"):
        for bad in (0, -64, 63):
            assert _norm(lib, **{name: bad}) == ALIGNMENT
    assert _norm(lib, rows=0, x=0, y=0, h=0x6000) == OK
    if not HAS_GPU:
        assert _norm(lib) in (CUDA, UNSUPPORTED)
        assert _norm(lib, x_out=0) in (CUDA, UNSUPPORTED)
        assert _norm(lib, y=0, post=0, pw=0, gate=0, x_out=0) in (CUDA, UNSUPPORTED)


# ------------------------------------------------------------------------------------ binding
def rows(T=5, Hk=2, H=4):
    return dict(q=dev(T, Hk, 128), k=dev(T, Hk, 128), v=dev(T, H, 128), g=dev(T, H, dtype=F32))


def prefill(stream=None, **kw):
    a = {**rows(), "cu_seqlens": dev(2, dtype=I32), **kw}
    return kda.lin_prefill(**a, stream=stream or Stream())


def decode(stream=None, **kw):
    a = {n: t.unsqueeze(0)[:, :4] for n, t in rows().items()}
    return kda.lin_decode(**{**a, "S_state": dev(1, 4, 128, 128, dtype=F32), **kw}, stream=stream or Stream())


def norm(stream=None, **kw):
    a = dict(x=dev(5, 64), weight=dev(64, dtype=F32), y=dev(5, 64), gate=dev(5, 64), post_weight=dev(64, dtype=F32))
    return kda.block_norm(**{**a, **kw}, stream=stream or Stream())


def test_binding_takes_sound_tensors(fakes):  # noqa: F811
    o, S = prefill()
    assert o.shape == (5, 4, 128) and o.dtype == BF and S.shape == (1, 4, 128, 128) and S.dtype == F32
    prefill(g=dev(4, dtype=F32), gate=dev(5, 4, 128), norm_weight=dev(128, dtype=F32), S_in=S, S_out=S, workspace=dev(512, dtype=torch.uint8))
    prefill(v=dev(5, 9, 128)[:, 1:5], gate=dev(7, 6, 128)[1:6, :4])
    o = decode()
    assert o.shape == (1, 4, 4, 128) and o.dtype == F32
    decode(g=dev(4, dtype=F32), n_commit=dev(1, dtype=I32))
    h, x = norm()
    assert h.dtype == x.dtype == BF and h.shape == x.shape == (5, 64)
    h, x = norm(x=dev(5, 64, dtype=F32))
    assert h.dtype == BF and x.dtype == F32
    a = dev(5, 64)
    assert norm(x=a, y=None, gate=None, post_weight=None)[1] is a
    norm(x=dev(5, 80)[:, :64], y=dev(5, 72)[:, 8:], x_out=dev(5, 64), h=dev(5, 64))


@pytest.mark.parametrize("call,name,bad", [
    (prefill, "q", dev(5, 2, 64)), (prefill, "q", dev(5, 128)), (prefill, "q", dev(5, 3, 128)), (prefill, "k", dev(5, 4, 128)),
    (prefill, "k", dev(6, 2, 128)), (prefill, "v", dev(4, 4, 128)), (prefill, "v", dev(5, 4, 256)[..., ::2]),
    (prefill, "g", dev(5, 2, dtype=F32)), (prefill, "g", dev(5, dtype=F32)), (prefill, "g", torch.zeros(5, 4)),
    (prefill, "cu_seqlens", dev(1, 2, dtype=I32)), (prefill, "S_in", dev(2, 4, 128, 128, dtype=F32)),
    (prefill, "S_in", dev(1, 4, 256, 128, dtype=F32)[:, :, ::2]), (prefill, "o", dev(5, 2, 128)),
    (prefill, "S_out", dev(1, 2, 128, 128, dtype=F32)), (prefill, "gate", dev(5, 2, 128)), (prefill, "norm_weight", dev(128, dtype=F32)),
    (prefill, "workspace", torch.zeros(512, dtype=torch.uint8)), (prefill, "workspace", dev(1024, dtype=torch.uint8)[::2]),
    (decode, "q", dev(1, 4, 2, 64)), (decode, "k", dev(1, 3, 2, 128)), (decode, "v", dev(2, 4, 4, 128)),
    (decode, "g", dev(1, 4, 2, dtype=F32)), (decode, "S_state", dev(1, 2, 128, 128, dtype=F32)),
    (decode, "n_commit", dev(2, dtype=I32)), (decode, "o", dev(1, 4, 2, 128, dtype=F32)),
    (norm, "x", dev(5, 4, 16)), (norm, "x", dev(5, 128)[:, ::2]), (norm, "y", dev(4, 64)), (norm, "y", dev(5, 72)),
    (norm, "gate", dev(5, 72)), (norm, "weight", dev(72, dtype=F32)), (norm, "post_weight", dev(63, dtype=F32)),
    (norm, "x_out", dev(5, 128)[:, :64]), (norm, "h", dev(4, 64)), (norm, "y", None),
])
def test_binding_refuses_bad_shapes(fakes, call, name, bad):  # noqa: F811
    with pytest.raises(ValueError):
        call(**{name: bad})


@pytest.mark.parametrize("call,name,bad", [
    (prefill, "q", dev(5, 2, 128, dtype=F32)), (prefill, "v", dev(5, 4, 128, dtype=torch.float16)), (prefill, "g", dev(5, 4)),
    (prefill, "g", [0.0]), (prefill, "cu_seqlens", dev(2, dtype=torch.int64)), (prefill, "S_in", dev(1, 4, 128, 128)),
    (prefill, "o", dev(5, 4, 128, dtype=F32)), (decode, "S_state", dev(1, 4, 128, 128)), (decode, "o", dev(1, 4, 4, 128)),
    (decode, "n_commit", dev(1, dtype=torch.int64)), (norm, "x", dev(5, 64, dtype=torch.float16)), (norm, "x", [1.0]),
    (norm, "y", dev(5, 64, dtype=F32)), (norm, "weight", dev(64)), (norm, "x_out", dev(5, 64, dtype=F32)), (norm, "h", dev(5, 64, dtype=F32)),
])
def test_binding_refuses_bad_types(fakes, call, name, bad):  # noqa: F811
    with pytest.raises(TypeError):
        call(**{name: bad})


@pytest.mark.parametrize("call", [prefill, decode, norm])
def test_what_a_call_makes_belongs_to_its_stream(fakes, call):  # noqa: F811
    s = Stream()
    NOTES.clear()
    call(stream=s)
    made = [n for n in NOTES if n[0] == "made on"]
    assert made and all(n[1] is s for n in made)
    assert ("kept for", "current") in NOTES


def test_another_device_is_refused(fakes):  # noqa: F811
    class Elsewhere(type(dev(1))):
        def get_device(self):
            return 1

    far = torch.zeros(5, 2, 128, dtype=BF).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="one device"):
        prefill(k=far)

    class There:
        cuda_stream = 1
        device = torch.device("cuda", 0)

    x = torch.zeros(5, 64, dtype=BF).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="not the device"):
        kda.block_norm(x, stream=There())
