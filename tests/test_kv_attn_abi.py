"""The attention cache's entry points reject bad arguments on the host, before any CUDA call,
and the binding rejects bad tensors (no GPU needed)."""
import ctypes

import pytest
import torch

import kimi_delta_attention_prefill_gb300 as kda
from kimi_delta_attention_prefill_gb300 import build

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5
HAS_GPU = torch.cuda.is_available()
P = ctypes.c_void_p


class KvCache(ctypes.Structure):  # kda_kv_cache
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3), ("k_scale_stride", ctypes.c_int64 * 2),
                ("v_scale_stride", ctypes.c_int64 * 2), ("n_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("dtype", ctypes.c_int)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.library()


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def cache(e4m3=False, heads=2, page=16, n_pages=8, **kw):
    row = [heads * page * 128, page * 128, 128]
    c = KvCache(k=0x100000, v=0x200000, k_stride=strides(*row), v_stride=strides(*row), n_pages=n_pages,
                     n_kv_heads=heads, page_size=page, dtype=int(e4m3))
    if e4m3:
        c.k_scale, c.v_scale = 0x300000, 0x400000
        c.k_scale_stride = c.v_scale_stride = strides(heads * page, page)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def _append(lib, c, k=0x1000, ks=(256, 128), d=128, T=5, n_seq=1, cu=0x2000, start=0x3000, table=0x4000, v=0x5000):
    return lib.kda_kv_append(ctypes.byref(c) if c else None, P(k), strides(*ks), P(v), strides(256, 128), P(table), n_seq, 4,
                             P(cu), P(start), T, d, None, None)


def _read(lib, c, k=0x1000, T=5, n_seq=1, cu=0x2000):
    return lib.kda_kv_read(ctypes.byref(c), P(k), P(0x5000), P(0x4000), n_seq, 4, P(cu), P(0x3000), T, 128, None, None)


def _prefill(lib, c, q=0x1000, qs=(512, 128), H=4, d=128, T=5, n_seq=1, cu=0x2000, scale=0.1, window=0, sink=0, o=0x6000,
             ws=0x700000, ws_bytes=1 << 40, max_pages=4, lse=None):
    return lib.kda_attn_prefill_paged(P(q), strides(*qs), ctypes.byref(c), P(0x4000), n_seq, max_pages, P(cu), P(0x3000), T,
                                      H, d, scale, window, sink, P(o), P(lse), P(ws), ws_bytes, None, None)


def _decode(lib, c, q=0x1000, qs=(512, 512, 128), H=4, d=128, B=3, n_tok=1, scale=0.1, window=0, sink=0, o=0x6000,
            ws=0x700000, ws_bytes=1 << 40, kv_len=0x3000):
    return lib.kda_attn_decode_paged(P(q), strides(*qs), ctypes.byref(c), P(0x4000), B, n_tok, 4, P(kv_len), H, d, scale,
                                     window, sink, P(o), None, P(ws), ws_bytes, None, None)


@pytest.mark.parametrize("call", [_append, _read, _prefill, _decode])
def test_cache_validation(lib, call):
    assert call(lib, cache(page=8)) == UNSUPPORTED
    assert call(lib, cache(page=48)) == UNSUPPORTED
    assert call(lib, cache(page=256)) == UNSUPPORTED
    assert call(lib, cache(dtype=2)) == UNSUPPORTED
    assert call(lib, cache(n_pages=-1)) == INVALID
    assert call(lib, cache(n_pages=1 << 31)) == INVALID
    assert call(lib, cache(n_kv_heads=0)) == INVALID
    assert call(lib, cache(k=0)) == INVALID
    assert call(lib, cache(e4m3=True, v_scale=0)) == INVALID
    assert call(lib, cache(k=0x100008)) == ALIGNMENT
    assert call(lib, cache(v_stride=strides(4096, 2048, 124))) == ALIGNMENT  # 248 bytes
    assert call(lib, cache(v_stride=strides(4096, 0, 128))) == ALIGNMENT
    assert call(lib, cache(v_stride=strides(-4096, 2048, 128))) == ALIGNMENT
    assert call(lib, cache(e4m3=True, k_stride=strides(4096, 2048, 136))) == ALIGNMENT
    assert call(lib, cache(e4m3=True, k_scale=0x300008)) == ALIGNMENT
    assert call(lib, cache(e4m3=True, k_scale_stride=strides(40, 16))) == ALIGNMENT
    if not HAS_GPU:
        assert call(lib, cache()) in (CUDA, UNSUPPORTED)
        assert call(lib, cache(e4m3=True, page=128)) in (CUDA, UNSUPPORTED)


def test_append_and_read_validation(lib):
    assert _append(lib, None) == INVALID
    assert _append(lib, cache(), d=64) == UNSUPPORTED
    assert _append(lib, cache(), T=-1) == INVALID
    assert _append(lib, cache(), n_seq=0) == INVALID
    assert _append(lib, cache(), T=0, n_seq=0) == OK and _append(lib, cache(), T=0) == OK
    assert _append(lib, cache(), k=0) == INVALID
    assert _append(lib, cache(), cu=0) == INVALID
    assert _append(lib, cache(), table=0) == INVALID
    assert _append(lib, cache(), k=0x1008) == ALIGNMENT
    assert _append(lib, cache(), ks=(260, 128)) == ALIGNMENT
    assert _append(lib, cache(), ks=(256, 0)) == ALIGNMENT
    assert _append(lib, cache(), start=0x3002) == ALIGNMENT
    assert _read(lib, cache(), k=0) == INVALID
    assert _read(lib, cache(), k=0x1004) == ALIGNMENT
    assert _read(lib, cache(), T=0) == OK


def test_attention_validation(lib):
    for call in (_prefill, _decode):
        assert call(lib, cache(), d=64) == UNSUPPORTED
        assert call(lib, cache(), H=3) == INVALID          # not a multiple of the kv heads
        assert call(lib, cache(), H=0) == INVALID
        assert call(lib, cache(), scale=float("nan")) == INVALID
        assert call(lib, cache(), scale=float("inf")) == INVALID
        assert call(lib, cache(), window=-1) == INVALID
        assert call(lib, cache(), sink=-1) == INVALID
        assert call(lib, cache(), q=0) == INVALID
        assert call(lib, cache(), o=0) == INVALID
        assert call(lib, cache(), q=0x1008) == ALIGNMENT
        assert call(lib, cache(), o=0x6004) == ALIGNMENT
        assert call(lib, cache(), ws=0x700010) == ALIGNMENT
        assert call(lib, cache(), ws=0) == WORKSPACE
        assert call(lib, cache(), ws_bytes=4096) == WORKSPACE
    assert _prefill(lib, cache(), qs=(508, 128)) == ALIGNMENT
    assert _prefill(lib, cache(), T=-1) == INVALID
    assert _prefill(lib, cache(), n_seq=0) == INVALID
    assert _prefill(lib, cache(), cu=0) == INVALID
    assert _prefill(lib, cache(), max_pages=1 << 28) == INVALID  # positions past 32 bits
    assert _prefill(lib, cache(), lse=0x6002) == ALIGNMENT
    assert _prefill(lib, cache(), T=0, n_seq=0) == OK
    assert _decode(lib, cache(), n_tok=0) == UNSUPPORTED
    assert _decode(lib, cache(), n_tok=5) == UNSUPPORTED
    assert _decode(lib, cache(), kv_len=0) == INVALID
    assert _decode(lib, cache(), B=0) == OK


def test_workspace_sizes(lib):
    """Parts of two partial items a block, whatever the lengths; bad shapes need none."""
    assert kda.attn_decode_workspace_size(4, 1, 8, 3) == 0
    assert kda.attn_decode_workspace_size(4, 5, 8, 2) == 0
    assert kda.attn_prefill_workspace_size(4, -1, 8, 2) == 0
    assert kda.attn_decode_workspace_size(4, 1, 8, 2) == kda.attn_decode_workspace_size(4000, 1, 8, 2) > 0
    assert kda.attn_prefill_workspace_size(1, 1 << 20, 8, 2) < 1 << 28


def test_binding_rejects_bad_tensors(lib):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kv_append(bf(4, 2, 128), bf(4, 2, 128), bf(3, 2, 16, 128), bf(3, 2, 16, 128), i32(1, 3), i32(2), i32(1))
    with pytest.raises(ValueError, match="n_pages"):
        kda.kv_read(bf(3, 2, 128), bf(3, 2, 128), i32(1, 3), i32(2), i32(1), 4)
    with pytest.raises(TypeError, match="bfloat16 or"):
        kda.attn_decode_paged(bf(1, 1, 2, 128), bf(3, 2, 16, 128).float(), bf(3, 2, 16, 128), i32(1, 3), i32(1))
