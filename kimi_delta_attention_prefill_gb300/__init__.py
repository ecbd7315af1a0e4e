"""GB300-native Kimi Delta Attention (KDA): chunkwise prefill and decode / verify.

Python binding of the C ABI in ``include/kda.h``: argument marshalling only.  Every
step of the computation runs in the CUDA kernels of ``libkda.so`` (sm_103a); there is
no CPU or PyTorch fallback, and a missing library raises ``KdaLibraryError``.

Functions mirror the C entry points: :func:`prefill` (``kda_prefill``, or
``kda_prefill_gated`` when gate logits are given), :func:`prefill_paged`
(``kda_prefill_paged``), :func:`prefill_host` (``kda_prefill_host``, host buffers),
:func:`decode` (``kda_decode``), :func:`decode_paged` (``kda_decode_paged``),
:func:`decode_fused` (``kda_decode_fused``), :func:`prefill_pairs` (``kda_prefill_pairs``),
:func:`combine_pairs` (``kda_combine_pairs``), :func:`prefill_noalloc`
(``kda_prefill_noalloc``), the attention cache's :func:`kv_append` (``kda_kv_append``),
:func:`kv_read` (``kda_kv_read``), :func:`attn_prefill_paged` (``kda_attn_prefill_paged``) and
:func:`attn_decode_paged` (``kda_attn_decode_paged``), linear attention's :func:`lin_prefill`
(``kda_lin_prefill``) and :func:`lin_decode` (``kda_lin_decode``), the step between blocks
:func:`block_norm` (``kda_block_norm``), the workspace-size queries, and
:func:`status_string` (``kda_status_string``).  The cross-device split's exchange is in :mod:`.kcp`.  Tensors are torch CUDA tensors (pinned
host tensors for :func:`prefill_host`); the launch goes to the current torch stream
unless ``stream`` is given.  Tensors that a call makes, outputs and workspaces, are made on the
stream that it runs on.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")
HEAD_DIM = 128
CHUNK = 64
MAX_DECODE_TOKENS = 4

_lib = None
_lock = threading.Lock()

_c_int, _c_i64, _c_sz, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p


class KdaLibraryError(RuntimeError):
    """The compiled CUDA library is missing or cannot be loaded."""


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


def library():
    """Load ``libkda.so`` (built by ``kimi_delta_attention_prefill_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise KdaLibraryError(
                    f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
            try:
                lib = ctypes.CDLL(LIB_PATH)
            except OSError as e:  # pragma: no cover - depends on the host
                raise KdaLibraryError(f"cannot load {LIB_PATH}: {e}") from e
            lib.kda_status_string.restype = ctypes.c_char_p
            lib.kda_status_string.argtypes = [_c_int]
            lib.kda_version.restype = _c_int
            lib.kda_version.argtypes = []
            lib.kda_decode.restype = _c_int
            lib.kda_decode.argtypes = [_vp] * 8 + [_c_int] * 4 + [_vp, _vp]
            lib.kda_prefill_workspace_size.restype = _c_sz
            lib.kda_prefill_workspace_size.argtypes = [_c_int, _c_int, _c_int, _c_i64, _c_int]
            lib.kda_prefill.restype = _c_int
            lib.kda_prefill.argtypes = ([_vp] * 7 + [_c_int, _c_i64] + [_vp, _vp, _c_i64] + [_vp] * 3 +
                                        [_c_int, _c_int, _c_int, _vp, _c_sz, _vp, _vp])
            lib.kda_prefill_gated.restype = _c_int
            lib.kda_prefill_gated.argtypes = ([_vp] * 7 + [ctypes.c_float] + [_vp, _vp] + [_c_int, _c_i64] +
                                              [_vp, _vp, _c_i64] + [_vp] * 3 +
                                              [_c_int, _c_int, _c_int, _vp, _c_sz, _vp, _vp])
            lib.kda_prefill_paged_workspace_size.restype = _c_sz
            lib.kda_prefill_paged_workspace_size.argtypes = [_c_int, _c_int, _c_int, _c_i64, _c_int, _c_i64]
            lib.kda_prefill_paged.restype = _c_int
            lib.kda_prefill_paged.argtypes = ([_vp] * 7 + [ctypes.c_float] + [_vp, _c_i64, _vp, _vp, _vp] +
                                              [_c_int, _c_i64, _vp, _vp, _c_i64, _vp, _vp] +
                                              [_c_int, _c_int, _c_int, _vp, _c_sz, _vp, _vp])
            lib.kda_decode_paged_workspace_size.restype = _c_sz
            lib.kda_decode_paged_workspace_size.argtypes = [_c_i64]
            lib.kda_decode_paged.restype = _c_int
            lib.kda_decode_paged.argtypes = ([_vp] * 6 + [_c_i64] + [_vp] * 4 + [_c_int] * 4 +
                                             [_vp, _c_sz, _vp, _vp])
            lib.kda_decode_fused.restype = _c_int
            lib.kda_decode_fused.argtypes = ([_vp] * 5 + [_c_int, _c_int] + [_vp, _vp, ctypes.c_float] + [_vp] * 3 +
                                             [ctypes.c_float] + [_vp] * 3 + [_c_int] * 4 + [_vp, _vp])
            lib.kda_prefill_host_workspace_size.restype = _c_sz
            lib.kda_prefill_host_workspace_size.argtypes = [_c_int, _c_int, _c_int, _c_i64, _c_i64]
            lib.kda_prefill_host.restype = _c_int
            lib.kda_prefill_host.argtypes = ([_vp] * 7 + [_c_int, _c_i64, _vp, _vp, _c_int, _c_int, _c_i64] +
                                             [_vp, _c_sz, _vp, _vp])
            lib.kda_prefill_host_blocks.restype = _c_int
            lib.kda_prefill_host_blocks.argtypes = [_vp, _c_int, _c_i64, _c_i64, _vp, _c_int]
            if hasattr(lib, "kda_debug_stall_next_prefill"):  # diagnostic hook (tests)
                lib.kda_debug_stall_next_prefill.restype = None
                lib.kda_debug_stall_next_prefill.argtypes = [_c_int]
            if hasattr(lib, "kda_debug_stall_next_attention"):  # diagnostic hook (tests)
                lib.kda_debug_stall_next_attention.restype = None
                lib.kda_debug_stall_next_attention.argtypes = [_c_int]
                lib.kda_debug_attention_kernel.restype = _c_int
                lib.kda_debug_attention_kernel.argtypes = [_c_int, _c_i64, _c_int, _c_int, _c_i64]
            if hasattr(lib, "kda_debug_stall_next_linear"):  # diagnostic hook (tests)
                lib.kda_debug_stall_next_linear.restype = None
                lib.kda_debug_stall_next_linear.argtypes = [_c_int]
            lib.kda_prefill_pairs.restype = _c_int
            lib.kda_prefill_pairs.argtypes = [_vp] * 6 + [_c_int, _c_i64, _vp, _vp, _c_int, _c_int, _vp, _vp]
            lib.kda_combine_pairs.restype = _c_int
            lib.kda_combine_pairs.argtypes = [_vp, _vp, _c_int, _vp, _vp, _c_int, _c_int, _c_int, _vp]
            lib.kda_prefill_noalloc.restype = _c_int
            lib.kda_prefill_noalloc.argtypes = ([_vp] * 7 + [_c_int, _c_i64] + [_vp, _vp, _c_i64] + [_vp] * 3 +
                                                [_c_int, _c_int, _c_int, _vp, _vp])
            cache = strides = _vp  # a kda_kv_cache, int64 arrays
            lib.kda_kv_append.restype = _c_int
            lib.kda_kv_append.argtypes = [cache, _vp, strides, _vp, strides, _vp, _c_int, _c_int, _vp, _vp, _c_i64,
                                          _c_int, _vp, _vp]
            lib.kda_kv_read.restype = _c_int
            lib.kda_kv_read.argtypes = [cache, _vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _c_i64, _c_int, _vp, _vp]
            lib.kda_attn_prefill_workspace_size.restype = _c_sz
            lib.kda_attn_prefill_workspace_size.argtypes = [_c_int, _c_i64, _c_int, _c_int, _c_int]
            lib.kda_attn_prefill_paged.restype = _c_int
            lib.kda_attn_prefill_paged.argtypes = ([_vp, strides, cache, _vp, _c_int, _c_int, _vp, _vp, _c_i64, _c_int,
                                                    _c_int, ctypes.c_float, _c_int, _c_int] +
                                                   [_vp, _vp, _vp, _c_sz, _vp, _vp])
            lib.kda_attn_decode_workspace_size.restype = _c_sz
            lib.kda_attn_decode_workspace_size.argtypes = [_c_int] * 5
            lib.kda_attn_decode_paged.restype = _c_int
            lib.kda_attn_decode_paged.argtypes = ([_vp, strides, cache, _vp, _c_int, _c_int, _c_int, _vp, _c_int, _c_int,
                                                   ctypes.c_float, _c_int, _c_int] + [_vp, _vp, _vp, _c_sz, _vp, _vp])
            rows = [_vp, strides] * 4 + [ctypes.c_float, _vp, strides, _vp, ctypes.c_float]  # q, k, v, g; output stage
            lib.kda_lin_prefill_workspace_size.restype = _c_sz
            lib.kda_lin_prefill_workspace_size.argtypes = [_c_int, _c_int, _c_int, _c_i64, _c_int]
            lib.kda_lin_prefill.restype = _c_int
            lib.kda_lin_prefill.argtypes = rows + [_vp, _vp, _c_int, _c_i64, _vp, _vp] + [_c_int] * 4 + [_vp, _c_sz, _vp, _vp]
            lib.kda_lin_decode.restype = _c_int
            lib.kda_lin_decode.argtypes = rows + [_vp, _vp, _vp] + [_c_int] * 5 + [_vp, _vp]
            lib.kda_block_norm.restype = _c_int
            lib.kda_block_norm.argtypes = [_vp, _c_int, _c_i64, _vp, _vp, _c_i64, _c_int, _vp, _vp, _c_i64, ctypes.c_float,
                                           ctypes.c_float, _vp, _vp, _c_i64, _c_int, _vp]
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().kda_status_string(int(status)).decode()


def version() -> int:
    return library().kda_version()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _scratch(n_bytes, device, stream):
    """A workspace for one call, made on the stream that the call runs on: the allocator must not give
    memory that another stream's work still uses, nor take it back before the call's kernels are done."""
    if stream is None:
        return torch.empty(n_bytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n_bytes, dtype=torch.uint8, device=device)


def _workspace(t):
    """Address and bytes of a workspace given by the caller (None: none)."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _output(shape, dtype, device, stream):
    """A call's output, made as :func:`_scratch`; the caller's stream may use it as well."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _need(t, name, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def decode(q, k, v, g, beta, S_state, n_commit=None, o=None, dev_status=None, stream=None):
    """One decode (n_tok = 1) or verify (n_tok <= 4) step; updates ``S_state`` in place.

    q, k, v ``[B, n_tok, H, 128]`` bf16; g ``[B, n_tok, H, 128]`` fp32; beta
    ``[B, n_tok, H]`` fp32; S_state ``[B, H, 128, 128]`` fp32; n_commit ``[B]`` int32 or
    None.  Returns o ``[B, n_tok, H, 128]`` fp32.
    """
    B, n_tok, H, d = q.shape
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, q.shape)
    _need(g, "g", torch.float32, q.shape)
    _need(beta, "beta", torch.float32, (B, n_tok, H))
    _need(S_state, "S_state", torch.float32, (B, H, d, d))
    if n_commit is not None:
        _need(n_commit, "n_commit", torch.int32, (B,))
    if o is None:
        o = _output((B, n_tok, H, d), torch.float32, q.device, stream)
    _need(o, "o", torch.float32, (B, n_tok, H, d))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    st = library().kda_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S_state), _ptr(n_commit),
                              _ptr(o), B, n_tok, H, d, _ptr(dev_status), _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_decode")
    return o


def decode_fused(qp, kp, vp, conv_w, conv_cache, z, a_log, b, S_state, n_commit=None, conv_act="none",
                 g_min=-5.0, gate=None, norm_weight=None, eps=1e-5, o=None, dev_status=None, stream=None):
    """A decode / verify step from projected inputs (``kda_decode_fused``): short causal
    convolution (``conv_w`` ``[3, H, 128, W]``, ``conv_cache`` ``[B, H, 3, W-1, 128]``, updated
    in place to the committed tokens), q / k L2 normalisation, alpha = exp(g_min
    sigmoid(e^a_log z)), beta = sigmoid(b), the recurrence on ``S_state`` (in place) and, with
    ``gate``, the output stage.  qp, kp, vp ``[B, n_tok, H, 128]`` bf16; z fp32 of the same
    shape; a_log ``[H]``; b ``[B, n_tok, H]``.  Returns o ``[B, n_tok, H, 128]`` fp32."""
    B, n_tok, H, d = qp.shape
    _need(qp, "qp", torch.bfloat16)
    _need(kp, "kp", torch.bfloat16, qp.shape)
    _need(vp, "vp", torch.bfloat16, qp.shape)
    _need(conv_w, "conv_w", torch.float32)
    if conv_w.dim() != 4 or tuple(conv_w.shape[:3]) != (3, H, d):
        raise ValueError(f"conv_w must have shape [3, {H}, {d}, W], got {tuple(conv_w.shape)}")
    W = conv_w.shape[3]
    if W > 1:
        _need(conv_cache, "conv_cache", torch.float32, (B, H, 3, W - 1, d))
    _need(z, "z", torch.float32, qp.shape)
    _need(a_log, "a_log", torch.float32, (H,))
    _need(b, "b", torch.float32, (B, n_tok, H))
    _need(S_state, "S_state", torch.float32, (B, H, d, d))
    if n_commit is not None:
        _need(n_commit, "n_commit", torch.int32, (B,))
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, qp.shape)
        if norm_weight is not None:
            _need(norm_weight, "norm_weight", torch.float32, (d,))
    if o is None:
        o = _output((B, n_tok, H, d), torch.float32, qp.device, stream)
    _need(o, "o", torch.float32, (B, n_tok, H, d))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    act = {"none": 0, "silu": 1}[conv_act]
    st = library().kda_decode_fused(_ptr(qp), _ptr(kp), _ptr(vp), _ptr(conv_w), _ptr(conv_cache) if W > 1 else None,
                                    W, act, _ptr(z), _ptr(a_log), float(g_min), _ptr(b), _ptr(gate),
                                    _ptr(norm_weight), float(eps), _ptr(S_state), _ptr(n_commit), _ptr(o), B, n_tok,
                                    H, d, _ptr(dev_status), _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_decode_fused")
    return o


def prefill_workspace_size(n_seq, H, total_tokens, n_segments=0, d=HEAD_DIM) -> int:
    return int(library().kda_prefill_workspace_size(int(n_seq), int(H), int(d), int(total_tokens),
                                                    int(n_segments)))


def prefill(q, k, v, g, beta, cu_seqlens, S_in=None, ckpt_off=None, ckpt_pos=None, o=None, S_out=None,
            ckpts=None, n_segments=0, workspace=None, dev_status=None, stream=None, gate=None,
            norm_weight=None, eps=1e-5):
    """Chunkwise prefill over packed sequences.

    q, k, v ``[T, H, 128]`` bf16; g ``[T, H, 128]`` fp32; beta ``[T, H]`` fp32;
    cu_seqlens ``[N+1]`` int32 (device); S_in ``[N, H, 128, 128]`` fp32 or None;
    ckpt_off ``[N+1]`` / ckpt_pos ``[n_ckpt]`` int32 (device) or None.
    With ``gate`` (``[T, H, 128]`` bf16 gate logits) the output stage is fused
    (``kda_prefill_gated``): the returned ``o`` holds
    ``sigmoid(gate) * norm_weight * o~ / sqrt(mean(o~^2) + eps)`` (``norm_weight`` ``[128]``
    fp32 or None for ones).
    Returns ``(o, S_out, ckpts)``.
    """
    T, H, d = q.shape
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, q.shape)
    _need(g, "g", torch.float32, q.shape)
    _need(beta, "beta", torch.float32, (T, H))
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    n_seq = cu_seqlens.shape[0] - 1
    if S_in is not None:
        _need(S_in, "S_in", torch.float32, (n_seq, H, d, d))
    n_ckpt = 0
    if ckpt_off is not None:
        _need(ckpt_off, "ckpt_off", torch.int32, (n_seq + 1,))
        _need(ckpt_pos, "ckpt_pos", torch.int32)
        n_ckpt = ckpt_pos.shape[0]
        if ckpts is None:
            ckpts = _output((n_ckpt, H, d, d), torch.float32, q.device, stream)
        _need(ckpts, "ckpts", torch.float32, (n_ckpt, H, d, d))
    if o is None:
        o = _output((T, H, d), torch.bfloat16, q.device, stream)
    _need(o, "o", torch.bfloat16, (T, H, d))
    if S_out is None:
        S_out = _output((n_seq, H, d, d), torch.float32, q.device, stream)
    _need(S_out, "S_out", torch.float32, (n_seq, H, d, d))
    ws_need = prefill_workspace_size(n_seq, H, T, n_segments, d)
    if workspace is None and ws_need > 0:
        workspace = _scratch(ws_need, q.device, stream)
    ws, ws_bytes = _workspace(workspace)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    if gate is None:
        st = library().kda_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S_in), _ptr(cu_seqlens),
                                   n_seq, T, _ptr(ckpt_off), _ptr(ckpt_pos), n_ckpt, _ptr(o), _ptr(S_out),
                                   _ptr(ckpts), H, d, int(n_segments), ws, ws_bytes, _ptr(dev_status),
                                   _stream_handle(stream))
        if st != 0:
            raise KdaError(st, "kda_prefill")
        return o, S_out, ckpts
    _need(gate, "gate", torch.bfloat16, q.shape)
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", torch.float32, (d,))
    st = library().kda_prefill_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(gate), _ptr(norm_weight),
                                     float(eps), _ptr(S_in), _ptr(cu_seqlens), n_seq, T, _ptr(ckpt_off),
                                     _ptr(ckpt_pos), n_ckpt, _ptr(o), _ptr(S_out), _ptr(ckpts), H, d,
                                     int(n_segments), ws, ws_bytes, _ptr(dev_status),
                                     _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_prefill_gated")
    return o, S_out, ckpts


def _pool(state_pool, d):
    _need(state_pool, "state_pool", torch.float32)
    if state_pool.dim() != 3 or tuple(state_pool.shape[1:]) != (d, d):
        raise ValueError(f"state_pool must have shape [n_pages, {d}, {d}], got {tuple(state_pool.shape)}")
    return state_pool.shape[0]


def _table(t, name, n):
    if t is not None:
        _need(t, name, torch.int32, (n,))
    return t


def prefill_paged_workspace_size(n_seq, H, total_tokens, n_pages, n_segments=0, d=HEAD_DIM) -> int:
    return int(library().kda_prefill_paged_workspace_size(int(n_seq), int(H), int(d), int(total_tokens),
                                                          int(n_segments), int(n_pages)))


def prefill_paged(q, k, v, g, beta, cu_seqlens, state_pool, s_in_page=None, s_out_page=None, ckpt_off=None,
                  ckpt_pos=None, ckpt_page=None, o=None, n_segments=0, workspace=None, dev_status=None,
                  stream=None, gate=None, norm_weight=None, eps=1e-5):
    """:func:`prefill` with every state in a page pool (``kda_prefill_paged``).

    state_pool ``[n_pages, 128, 128]`` fp32; s_in_page / s_out_page ``[N * H]`` int32
    (entry ``seq * H + h``; -1 = zeros / not written; None = all zeros / none); ckpt_page
    ``[n_ckpt * H]`` int32 (entry ``j * H + h``).  A call never writes a page it reads
    (except a unit's own final state in place) and writes each page once; a violation
    writes nothing and sets ``dev_status`` to KDA_ERR_DEVICE_CHECK.  Returns ``o``.
    """
    T, H, d = q.shape
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, q.shape)
    _need(g, "g", torch.float32, q.shape)
    _need(beta, "beta", torch.float32, (T, H))
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    n_seq = cu_seqlens.shape[0] - 1
    n_pages = _pool(state_pool, d)
    _table(s_in_page, "s_in_page", n_seq * H)
    _table(s_out_page, "s_out_page", n_seq * H)
    n_ckpt = 0
    if ckpt_off is not None:
        _need(ckpt_off, "ckpt_off", torch.int32, (n_seq + 1,))
        _need(ckpt_pos, "ckpt_pos", torch.int32)
        n_ckpt = ckpt_pos.shape[0]
        _table(ckpt_page, "ckpt_page", n_ckpt * H)
    if o is None:
        o = _output((T, H, d), torch.bfloat16, q.device, stream)
    _need(o, "o", torch.bfloat16, (T, H, d))
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, q.shape)
        if norm_weight is not None:
            _need(norm_weight, "norm_weight", torch.float32, (d,))
    if workspace is None:
        need = prefill_paged_workspace_size(n_seq, H, T, n_pages, n_segments, d)
        workspace = _scratch(need, q.device, stream)
    ws, ws_bytes = _workspace(workspace)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    st = library().kda_prefill_paged(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(gate), _ptr(norm_weight),
                                     float(eps), _ptr(state_pool), n_pages, _ptr(s_in_page), _ptr(s_out_page),
                                     _ptr(cu_seqlens), n_seq, T, _ptr(ckpt_off), _ptr(ckpt_pos), n_ckpt,
                                     _ptr(ckpt_page), _ptr(o), H, d, int(n_segments), ws, ws_bytes,
                                     _ptr(dev_status), _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_prefill_paged")
    return o


def decode_paged_workspace_size(n_pages) -> int:
    return int(library().kda_decode_paged_workspace_size(int(n_pages)))


def decode_paged(q, k, v, g, beta, state_pool, s_in_page, s_out_page=None, n_commit=None, o=None, workspace=None,
                 dev_status=None, stream=None):
    """:func:`decode` with the states in a page pool (``kda_decode_paged``).

    s_in_page ``[B * H]`` int32 (entry ``b * H + h``; -1 = a zero state); s_out_page the
    same, or None to update in place.  A destination other than the source receives the
    state after ``n_commit[b]`` tokens (the entry state when that is 0).  Returns ``o``.
    """
    B, n_tok, H, d = q.shape
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, q.shape)
    _need(g, "g", torch.float32, q.shape)
    _need(beta, "beta", torch.float32, (B, n_tok, H))
    n_pages = _pool(state_pool, d)
    _need(s_in_page, "s_in_page", torch.int32, (B * H,))
    _table(s_out_page, "s_out_page", B * H)
    if n_commit is not None:
        _need(n_commit, "n_commit", torch.int32, (B,))
    if o is None:
        o = _output((B, n_tok, H, d), torch.float32, q.device, stream)
    _need(o, "o", torch.float32, (B, n_tok, H, d))
    if workspace is None:
        workspace = _scratch(decode_paged_workspace_size(n_pages), q.device, stream)
    ws, ws_bytes = _workspace(workspace)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    st = library().kda_decode_paged(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool), n_pages,
                                    _ptr(s_in_page), _ptr(s_out_page), _ptr(n_commit), _ptr(o), B, n_tok, H, d,
                                    ws, ws_bytes, _ptr(dev_status), _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_decode_paged")
    return o


def _host(t, name, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def prefill_host_blocks(cu_seqlens, block_tokens=0):
    """The block borders of :func:`prefill_host` for a host ``cu_seqlens`` (a list)."""
    _host(cu_seqlens, "cu_seqlens", torch.int32)
    n_seq = cu_seqlens.shape[0] - 1
    T = int(cu_seqlens[-1]) if n_seq >= 0 else 0
    out = torch.zeros(66, dtype=torch.int64)
    n = library().kda_prefill_host_blocks(_ptr(cu_seqlens), n_seq, T, int(block_tokens), _ptr(out), 66)
    if n < 0:
        raise ValueError("bad packing, block size, or more than 64 blocks")
    return out[:n + 1].tolist() if n > 0 else []


def prefill_host_workspace_size(n_seq, H, total_tokens, block_tokens=0, d=HEAD_DIM) -> int:
    return int(library().kda_prefill_host_workspace_size(int(n_seq), int(H), int(d), int(total_tokens),
                                                         int(block_tokens)))


def prefill_host(q, k, v, g, beta, cu_seqlens, S_in=None, o=None, S_out=None, block_tokens=0, workspace=None,
                 dev_status=None, stream=None):
    """:func:`prefill` from host tensors (``kda_prefill_host``): uploads, computes and downloads
    in pipelined blocks.  q, k, v, g, beta, S_in, o, S_out are HOST tensors (pinned for
    overlap); cu_seqlens a host int32 tensor.  ``workspace`` is a device uint8 tensor (made
    here when absent).  Returns ``(o, S_out)``; they are complete once ``stream`` is
    synchronised."""
    T, H, d = q.shape
    _host(q, "q", torch.bfloat16)
    _host(k, "k", torch.bfloat16, q.shape)
    _host(v, "v", torch.bfloat16, q.shape)
    _host(g, "g", torch.float32, q.shape)
    _host(beta, "beta", torch.float32, (T, H))
    _host(cu_seqlens, "cu_seqlens", torch.int32)
    n_seq = cu_seqlens.shape[0] - 1
    if S_in is not None:
        _host(S_in, "S_in", torch.float32, (n_seq, H, d, d))
    if o is None:
        o = torch.empty((T, H, d), dtype=torch.bfloat16).pin_memory()
    _host(o, "o", torch.bfloat16, (T, H, d))
    if S_out is None:
        S_out = torch.empty((n_seq, H, d, d), dtype=torch.float32).pin_memory()
    _host(S_out, "S_out", torch.float32, (n_seq, H, d, d))
    dev = torch.device("cuda", torch.cuda.current_device()) if stream is None else stream.device
    if workspace is None:
        workspace = _scratch(prefill_host_workspace_size(n_seq, H, T, block_tokens, d), dev, stream)
    _need(workspace, "workspace", torch.uint8)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    st = library().kda_prefill_host(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S_in), _ptr(cu_seqlens),
                                    n_seq, T, _ptr(o), _ptr(S_out), H, d, int(block_tokens), _ptr(workspace),
                                    workspace.numel(), _ptr(dev_status), _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_prefill_host")
    return o, S_out


def debug_stall_next_prefill(chunk):
    """Test hook (``kda_debug_stall_next_prefill``): the next prefill launch withholds one
    hand-off at ``chunk`` and gives up its waits after 4096 polls, so it reports
    KDA_ERR_TIMEOUT in ``dev_status`` without any fault."""
    library().kda_debug_stall_next_prefill(int(chunk))


def debug_stall_next_attention(copy):
    """Test hook (``kda_debug_stall_next_attention``): in the next attention call each block leaves
    out one copy of its keys; the call reports KDA_ERR_TIMEOUT in ``dev_status`` after some
    seconds, without any fault."""
    library().kda_debug_stall_next_attention(int(copy))


def debug_stall_next_linear(copy):
    """Test hook (``kda_debug_stall_next_linear``): in the next :func:`lin_prefill` call each block
    leaves out one copy; the call reports KDA_ERR_TIMEOUT in ``dev_status``, without any fault."""
    library().kda_debug_stall_next_linear(int(copy))


def debug_attention_kernel(n_seq, total_tokens, H, n_kv_heads, most_keys) -> int:
    """Which kernel an :func:`attn_prefill_paged` call takes (``kda_debug_attention_kernel``): 1 the
    tensor-core kernel, 0 the warp-level one.  ``most_keys`` is the page table's width in tokens."""
    return int(library().kda_debug_attention_kernel(int(n_seq), int(total_tokens), int(H), int(n_kv_heads), int(most_keys)))


NOALLOC_SCRATCH_BYTES = 32 << 20


def prefill_noalloc(q, k, v, g, beta, cu_seqlens, S_in=None, ckpt_off=None, ckpt_pos=None, o=None, S_out=None,
                    ckpts=None, n_segments=0, dev_status=None, stream=None):
    """:func:`prefill` for callers that cannot allocate device memory (``kda_prefill_noalloc``).

    The library takes its scratch from a fixed 32 MiB array of its own instead of a
    caller-provided workspace; larger problems raise ``KdaError`` (KDA_ERR_WORKSPACE).
    Output tensors are created here only when not given; pass them in to allocate nothing.
    Calls share the array: do not let two of them overlap on the GPU.
    """
    T, H, d = q.shape
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, q.shape)
    _need(g, "g", torch.float32, q.shape)
    _need(beta, "beta", torch.float32, (T, H))
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    n_seq = cu_seqlens.shape[0] - 1
    if S_in is not None:
        _need(S_in, "S_in", torch.float32, (n_seq, H, d, d))
    n_ckpt = 0
    if ckpt_off is not None:
        _need(ckpt_off, "ckpt_off", torch.int32, (n_seq + 1,))
        _need(ckpt_pos, "ckpt_pos", torch.int32)
        n_ckpt = ckpt_pos.shape[0]
        if ckpts is None:
            ckpts = _output((n_ckpt, H, d, d), torch.float32, q.device, stream)
        _need(ckpts, "ckpts", torch.float32, (n_ckpt, H, d, d))
    if o is None:
        o = _output((T, H, d), torch.bfloat16, q.device, stream)
    _need(o, "o", torch.bfloat16, (T, H, d))
    if S_out is None:
        S_out = _output((n_seq, H, d, d), torch.float32, q.device, stream)
    _need(S_out, "S_out", torch.float32, (n_seq, H, d, d))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    st = library().kda_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S_in),
                                       _ptr(cu_seqlens), n_seq, T, _ptr(ckpt_off), _ptr(ckpt_pos), n_ckpt, _ptr(o),
                                       _ptr(S_out), _ptr(ckpts), H, d, int(n_segments), _ptr(dev_status),
                                       _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_prefill_noalloc")
    return o, S_out, ckpts


def prefill_pairs(q, k, v, g, beta, cu_seqlens, M=None, S_tilde=None, dev_status=None, stream=None):
    """Per (sequence, head), the pair (M, S~) of the sequence's rows (``kda_prefill_pairs``):
    the cumulative transition and the state from a zero entry state.  Inputs as
    :func:`prefill`.  Returns ``(M, S_tilde)``, each ``[N, H, 128, 128]`` fp32."""
    T, H, d = q.shape
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, q.shape)
    _need(g, "g", torch.float32, q.shape)
    _need(beta, "beta", torch.float32, (T, H))
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    n_seq = cu_seqlens.shape[0] - 1
    if M is None:
        M = _output((n_seq, H, d, d), torch.float32, q.device, stream)
    if S_tilde is None:
        S_tilde = _output((n_seq, H, d, d), torch.float32, q.device, stream)
    _need(M, "M", torch.float32, (n_seq, H, d, d))
    _need(S_tilde, "S_tilde", torch.float32, (n_seq, H, d, d))
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32)
    st = library().kda_prefill_pairs(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), n_seq, T,
                                     _ptr(M), _ptr(S_tilde), H, d, _ptr(dev_status), _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_prefill_pairs")
    return M, S_tilde


def combine_pairs(M, S_tilde, S_in=None, entry=None, stream=None):
    """Entry states after the ranges whose pairs are given (``kda_combine_pairs``): M and
    S_tilde ``[R, N, H, 128, 128]`` fp32 (R >= 0), S_in ``[N, H, 128, 128]`` or None (zeros).
    Returns ``entry`` ``[N, H, 128, 128]``: E = S_in, then E = S~_r + M_r E for r = 0 .. R-1."""
    _need(M, "M", torch.float32)
    if M.dim() != 5:
        raise ValueError(f"M must have shape [R, N, H, d, d], got {tuple(M.shape)}")
    R, n_seq, H, d, _ = M.shape
    _need(S_tilde, "S_tilde", torch.float32, M.shape)
    if S_in is not None:
        _need(S_in, "S_in", torch.float32, (n_seq, H, d, d))
    if entry is None:
        entry = _output((n_seq, H, d, d), torch.float32, M.device, stream)
    _need(entry, "entry", torch.float32, (n_seq, H, d, d))
    st = library().kda_combine_pairs(_ptr(M) if R else None, _ptr(S_tilde) if R else None, R, _ptr(S_in),
                                     _ptr(entry), n_seq, H, d, _stream_handle(stream))
    if st != 0:
        raise KdaError(st, "kda_combine_pairs")
    return entry


# ------------------------------------------------------------------------ attention cache
# A decode step makes a few of these calls a layer and each runs for microseconds, so what is
# checked for every call is checked in as few steps as Python allows; the functions that say what
# is wrong run only when something is.
_BF16, _E4M3, _I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32
_pack_cache = struct.Struct("4q 3q 3q 2q 2q q 3i 4x").pack  # kda_kv_cache
_pack2, _pack3, _pack4 = (struct.Struct(n).pack for n in ("2q", "3q", "4q"))
_ALIGNMENT = 3  # KDA_ERR_ALIGNMENT
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(_current_device())
    return _stream_handle(stream)


def _say_rows(t, name, dtype, lead):
    """Why ``t`` is not a tensor ``lead + [128]`` of rows; None: it is."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = tuple(lead) + (HEAD_DIM,)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _sound(shape, strides):
    """Strides of all dimensions but the last.  torch gives dimensions of extent 1 (and those of
    empty tensors) any stride; the library wants a sound one."""
    lead = shape[:-1]
    for s in strides[:-1]:
        if s <= 0 or s & 15:
            break
    else:
        return strides[:-1]
    if 1 not in lead and 0 not in lead:
        return strides[:-1]  # the library says what is wrong with them
    packed = [1] * len(shape)
    for i in range(len(shape) - 2, -1, -1):
        packed[i] = packed[i + 1] * max(shape[i + 1], 1)
    empty = 0 in lead
    return tuple(p if empty or n == 1 else s for p, s, n in zip(packed, strides, lead))


def _rows_of(t, name, lead):
    """Strides of bf16 rows ``lead + [128]``; all dimensions but the last may be strided."""
    try:
        shape, strides = t.shape, t.stride()
        good = shape == lead + (HEAD_DIM,) and t.dtype is _BF16 and t.is_cuda and strides[-1] == 1
    except AttributeError:
        good = False
    if not good:
        _say_rows(t, name, _BF16, lead)
        shape, strides = t.shape, t.stride()
    return _sound(shape, strides)


def _say_cache(k_pool, v_pool, k_scale, v_scale):
    if not isinstance(k_pool, torch.Tensor) or k_pool.dim() != 4:
        raise ValueError("k_pool must be a tensor [n_pages, n_kv_heads, page_size, 128]")
    if k_pool.dtype not in (_BF16, _E4M3):
        raise TypeError(f"k_pool must be torch.bfloat16 or torch.float8_e4m3fn, got {k_pool.dtype}")
    lead = tuple(k_pool.shape[:3])
    _say_rows(k_pool, "k_pool", k_pool.dtype, lead)
    _say_rows(v_pool, "v_pool", k_pool.dtype, lead)
    if k_pool.dtype == _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale / v_scale belong to a float8_e4m3fn cache")
        return
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is None:
            raise ValueError(f"{name} is required for a float8_e4m3fn cache")
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.uint8:
            raise TypeError(f"{name} must be torch.uint8, got {t.dtype}")
        if tuple(t.shape) != lead:
            raise ValueError(f"{name} must have shape {lead}, got {tuple(t.shape)}")
        if t.numel() and t.stride(-1) != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")


def _kv_cache(k_pool, v_pool, k_scale, v_scale):
    """The cache as the library takes it (the bytes of a kda_kv_cache), and its heads."""
    try:
        shape, dtype, ks, vs = k_pool.shape, k_pool.dtype, k_pool.stride(), v_pool.stride()
        good = (len(shape) == 4 and shape[3] == HEAD_DIM and v_pool.shape == shape and v_pool.dtype is dtype
                and k_pool.is_cuda and v_pool.is_cuda and ks[3] == 1 and vs[3] == 1)
        if dtype is _E4M3:
            lead = shape[:3]
            good = (good and k_scale.shape == lead and v_scale.shape == lead and k_scale.dtype is torch.uint8
                    and v_scale.dtype is torch.uint8 and k_scale.is_cuda and v_scale.is_cuda)
            kss, vss = k_scale.stride(), v_scale.stride()
            good = good and kss[2] == 1 and vss[2] == 1
        else:
            good = good and dtype is _BF16 and k_scale is None and v_scale is None
    except (AttributeError, IndexError):
        good = False
    if not good:
        _say_cache(k_pool, v_pool, k_scale, v_scale)
        shape, dtype, ks, vs = k_pool.shape, k_pool.dtype, k_pool.stride(), v_pool.stride()
        if dtype is _E4M3:
            lead, kss, vss = shape[:3], k_scale.stride(), v_scale.stride()
    ks, vs = _sound(shape, ks), _sound(shape, vs)
    n, heads, page, _ = shape
    if dtype is _E4M3:
        return _pack_cache(k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *ks, *vs,
                           *_sound(lead, kss), *_sound(lead, vss), n, heads, page, 1), heads
    return _pack_cache(k_pool.data_ptr(), v_pool.data_ptr(), 0, 0, *ks, *vs, 0, 0, 0, 0, n, heads, page, 0), heads


def _index(t, name, shape):
    """Address of a contiguous int32 CUDA tensor of that shape."""
    try:
        if t.dtype is _I32 and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, _I32, shape)
    return t.data_ptr()


def _page_table(page_table):
    try:
        shape = page_table.shape
        if len(shape) == 2 and page_table.dtype is _I32 and page_table.is_cuda and page_table.is_contiguous():
            return shape
    except AttributeError:
        pass
    _need(page_table, "page_table", _I32)
    if page_table.dim() != 2:
        raise ValueError(f"page_table must have shape [sequences, pages], got {tuple(page_table.shape)}")
    return page_table.shape


def _status_ptr(dev_status):
    return None if dev_status is None else _need(dev_status, "dev_status", _I32).data_ptr()


def kv_append(k, v, k_pool, v_pool, page_table, cu_seqlens, kv_start, k_scale=None, v_scale=None, dev_status=None,
              stream=None):
    """Write new tokens' keys and values into the paged attention cache (``kda_kv_append``).

    k, v ``[T, Hkv, 128]`` bf16, packed over sequences (token and head dimensions may be
    strided); k_pool, v_pool ``[n_pages, Hkv, page_size, 128]`` bf16 or float8_e4m3fn (any
    strides over the first three dimensions; page_size 16, 32, 64 or 128), with k_scale,
    v_scale ``[n_pages, Hkv, page_size]`` uint8 for float8_e4m3fn: a row's values are
    ``code * 2**(scale - 127)``, scale 255 marks a row of NaN (a cache filled by others: scales
    47 to 207, see ``kda.h``).  page_table ``[N, max_pages]``
    int32 (-1: tokens there are not written); cu_seqlens ``[N + 1]``, kv_start ``[N]`` int32:
    row ``cu[i] + t`` becomes token ``kv_start[i] + t`` of sequence i.  Updates the pools (and
    scales) in place.
    """
    c, heads = _kv_cache(k_pool, v_pool, k_scale, v_scale)
    n_seq, max_pages = _page_table(page_table)
    T = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    ks, vs = _rows_of(k, "k", (T, heads)), _rows_of(v, "v", (T, heads))
    st = (_lib or library()).kda_kv_append(
        c, k.data_ptr(), _pack2(*ks), v.data_ptr(), _pack2(*vs), page_table.data_ptr(), n_seq, max_pages,
        _index(cu_seqlens, "cu_seqlens", (n_seq + 1,)), _index(kv_start, "kv_start", (n_seq,)), T, HEAD_DIM,
        _status_ptr(dev_status), _stream_of(stream))
    if st != 0:
        raise KdaError(st, "kda_kv_append")


def kv_read(k_pool, v_pool, page_table, cu_seqlens, kv_start, total_tokens, k_scale=None, v_scale=None, k=None, v=None,
            dev_status=None, stream=None):
    """Read ranges of cached tokens back as packed bf16 rows (``kda_kv_read``).

    Rows ``cu[i] .. cu[i + 1]`` of the result are tokens ``kv_start[i] ..`` of sequence i;
    ``total_tokens`` is ``cu[N]``.  The cache's arguments are those of :func:`kv_append`.
    Returns ``(k, v)``, each ``[total_tokens, Hkv, 128]`` bf16 (float8 values are exact in bf16).
    """
    c, heads = _kv_cache(k_pool, v_pool, k_scale, v_scale)
    n_seq, max_pages = _page_table(page_table)
    T = int(total_tokens)
    shape = (T, heads, HEAD_DIM)
    k = _output(shape, _BF16, k_pool.device, stream) if k is None else _need(k, "k", _BF16, shape)
    v = _output(shape, _BF16, k_pool.device, stream) if v is None else _need(v, "v", _BF16, shape)
    st = (_lib or library()).kda_kv_read(
        c, k.data_ptr(), v.data_ptr(), page_table.data_ptr(), n_seq, max_pages,
        _index(cu_seqlens, "cu_seqlens", (n_seq + 1,)), _index(kv_start, "kv_start", (n_seq,)), T, HEAD_DIM,
        _status_ptr(dev_status), _stream_of(stream))
    if st != 0:
        raise KdaError(st, "kda_kv_read")
    return k, v


def attn_prefill_workspace_size(n_seq, total_tokens, H, n_kv_heads, d=HEAD_DIM) -> int:
    return int(library().kda_attn_prefill_workspace_size(int(n_seq), int(total_tokens), int(H), int(n_kv_heads), int(d)))


def attn_decode_workspace_size(B, n_tok, H, n_kv_heads, d=HEAD_DIM) -> int:
    return int(library().kda_attn_decode_workspace_size(int(B), int(n_tok), int(H), int(n_kv_heads), int(d)))


def _c_count(n):
    """A window or a number of tokens as the library's 32-bit int: more than fits is more than any
    sequence has, and what is negative stays so."""
    return max(-1, min(n, 0x7fffffff))


def _attn_outputs(q, shape, o, lse, return_lse, stream):
    o = _output(shape, _BF16, q.device, stream) if o is None else _need(o, "o", _BF16, shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, shape[:-1])
    elif return_lse:
        lse = _output(shape[:-1], torch.float32, q.device, stream)
    return o, lse


def attn_prefill_paged(q, k_pool, v_pool, page_table, cu_seqlens, kv_len, k_scale=None, v_scale=None, scale=None,
                       window=0, n_sink=0, o=None, lse=None, return_lse=False, workspace=None, dev_status=None,
                       stream=None):
    """Causal attention of a chunk of new tokens over the paged cache (``kda_attn_prefill_paged``).

    q ``[T, H, 128]`` bf16, packed over sequences (token and head dimensions may be strided; H a
    multiple of the cache's heads); the cache as in :func:`kv_append`, the new tokens already in
    it; cu_seqlens ``[N + 1]`` int32; kv_len ``[N]`` int32 the tokens in the cache, new ones
    included.  ``scale`` defaults to 1 / sqrt(128).  With ``window`` > 0 a token sees the last
    ``window`` keys up to itself and the first ``n_sink`` of the sequence.  Returns o
    ``[T, H, 128]`` bf16, or ``(o, lse)`` with ``return_lse`` or ``lse`` given (``[T, H]`` fp32).
    """
    c, heads = _kv_cache(k_pool, v_pool, k_scale, v_scale)
    n_seq, max_pages = _page_table(page_table)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [T, H, 128]")
    shape = q.shape
    T, H, _ = shape
    qs = _rows_of(q, "q", (T, H))
    o, lse = _attn_outputs(q, shape, o, lse, return_lse, stream)
    lib = _lib or library()
    if workspace is None:
        ws_bytes = lib.kda_attn_prefill_workspace_size(n_seq, T, H, heads, HEAD_DIM)
        workspace = _scratch(ws_bytes, q.device, stream)
        ws = workspace.data_ptr()
    else:
        ws, ws_bytes = _workspace(workspace)
    st = lib.kda_attn_prefill_paged(
        q.data_ptr(), _pack2(*qs), c, page_table.data_ptr(), n_seq, max_pages,
        _index(cu_seqlens, "cu_seqlens", (n_seq + 1,)), _index(kv_len, "kv_len", (n_seq,)), T, H, HEAD_DIM,
        HEAD_DIM ** -0.5 if scale is None else scale, _c_count(window), _c_count(n_sink), o.data_ptr(),
        None if lse is None else lse.data_ptr(), ws, ws_bytes, _status_ptr(dev_status), _stream_of(stream))
    if st != 0:
        raise KdaError(st, "kda_attn_prefill_paged")
    return o if lse is None else (o, lse)


def attn_decode_paged(q, k_pool, v_pool, page_table, kv_len, k_scale=None, v_scale=None, scale=None, window=0, n_sink=0,
                      o=None, lse=None, return_lse=False, workspace=None, dev_status=None, stream=None):
    """:func:`attn_prefill_paged` for a decode or verify step (``kda_attn_decode_paged``): q
    ``[B, n_tok, H, 128]`` bf16 with n_tok <= 4, the last n_tok tokens of each sequence; kv_len
    ``[B]`` int32 includes them (0: an idle slot, o = 0).  Returns o ``[B, n_tok, H, 128]``
    bf16, or ``(o, lse)`` with lse ``[B, n_tok, H]`` fp32.
    """
    c, heads = _kv_cache(k_pool, v_pool, k_scale, v_scale)
    n_seq, max_pages = _page_table(page_table)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor [B, n_tok, H, 128]")
    shape = q.shape
    B, n_tok, H, _ = shape
    qs = _rows_of(q, "q", (B, n_tok, H))
    if B != n_seq:
        raise ValueError(f"page_table must have {B} rows, got {n_seq}")
    o, lse = _attn_outputs(q, shape, o, lse, return_lse, stream)
    lib = _lib or library()
    if workspace is None:
        ws_bytes = lib.kda_attn_decode_workspace_size(B, n_tok, H, heads, HEAD_DIM)
        workspace = _scratch(ws_bytes, q.device, stream)
        ws = workspace.data_ptr()
    else:
        ws, ws_bytes = _workspace(workspace)
    st = lib.kda_attn_decode_paged(
        q.data_ptr(), _pack3(*qs), c, page_table.data_ptr(), B, n_tok, max_pages, _index(kv_len, "kv_len", (B,)), H,
        HEAD_DIM, HEAD_DIM ** -0.5 if scale is None else scale, _c_count(window), _c_count(n_sink), o.data_ptr(),
        None if lse is None else lse.data_ptr(), ws, ws_bytes, _status_ptr(dev_status), _stream_of(stream))
    if st != 0:
        raise KdaError(st, "kda_attn_decode_paged")
    return o if lse is None else (o, lse)


# ---------------------------------------------------- linear attention with a decay a head
_F32 = torch.float32


def _on(device, stream, *tensors):
    """All tensors are on one device, and it is the one that the call runs on.  What is no tensor is refused by name
    where its type is looked at."""
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.get_device() != device:
            raise ValueError(f"all tensors must be on one device, got cuda:{device} and {t.device}")
    if device >= 0 and device != _here(stream):
        raise ValueError(f"the tensors are on cuda:{device}, which is not the device that the call runs on")


def _here(stream):
    """The device that the call runs on."""
    return _current_device() if stream is None else stream.device.index


def _decays(g, lead, H):
    """Strides of the log-decays: ``lead + [H]``, or ``[H]`` for every token alike."""
    if not isinstance(g, torch.Tensor):
        raise TypeError("g must be a torch.Tensor")
    if not g.is_cuda:
        raise ValueError("g must be a CUDA tensor")
    if g.dtype is not _F32:
        raise TypeError(f"g must be {_F32}, got {g.dtype}")
    if g.shape == lead + (H,):
        return g.stride()
    if g.shape == (H,):
        return (0,) * len(lead) + g.stride()
    raise ValueError(f"g must have shape {lead + (H,)} or {(H,)}, got {tuple(g.shape)}")


def _stage_rows(gate, norm_weight, shape, dev, pack):
    """(whether they are what they should be at a quick look, gate's strides)"""
    if gate is None:
        return norm_weight is None, None
    if gate.shape != shape:
        return False, None  # its strides may be any number
    st = gate.stride()
    return (gate.dtype is _BF16 and gate.get_device() == dev and st[-1] == 1
            and (norm_weight is None or (norm_weight.shape == (HEAD_DIM,) and norm_weight.dtype is _F32
                                         and norm_weight.get_device() == dev and norm_weight.is_contiguous()))), pack(*st)


def _say_lin_rows(q, k, v, g, gate, norm_weight, n_lead, names, pack):
    """What the two calls share: sizes, and the rows' strides as the library takes them; says what is wrong.  The calls
    look at well-formed arguments in fewer steps, as for the attention cache, and come here with the others: torch gives
    dimensions of extent 1 any stride, which the library may refuse."""
    if not isinstance(q, torch.Tensor) or q.dim() != n_lead + 2:
        raise ValueError(f"q must be a tensor [{names}, heads, {HEAD_DIM}]")
    if not isinstance(v, torch.Tensor) or v.dim() != n_lead + 2:
        raise ValueError(f"v must be a tensor [{names}, heads, {HEAD_DIM}]")
    shape = q.shape
    lead, Hk, H = tuple(shape[:n_lead]), shape[n_lead], v.shape[n_lead]
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"the heads of v must be a multiple of those of q and k, got {H} and {Hk}")
    qs, ks = _rows_of(q, "q", lead + (Hk,)), _rows_of(k, "k", lead + (Hk,))
    vs, gs = _rows_of(v, "v", lead + (H,)), _decays(g, lead, H)
    gates = None
    if gate is not None:
        gates = pack(*_rows_of(gate, "gate", lead + (H,)))
        if norm_weight is not None:
            _need(norm_weight, "norm_weight", _F32, (HEAD_DIM,))
    elif norm_weight is not None:
        raise ValueError("norm_weight belongs to the output stage, which needs gate")
    return lead, Hk, H, pack(*qs), pack(*ks), pack(*vs), pack(*gs), gates


def lin_prefill_workspace_size(n_seq, H, total_tokens, n_segments=0, d=HEAD_DIM) -> int:
    return int(library().kda_lin_prefill_workspace_size(int(n_seq), int(H), int(d), int(total_tokens), int(n_segments)))


def lin_prefill(q, k, v, g, cu_seqlens, S_in=None, scale=1.0, gate=None, norm_weight=None, eps=1e-5, o=None, S_out=None,
                n_segments=0, workspace=None, dev_status=None, stream=None):
    """Linear attention with a decay a head over packed sequences (``kda_lin_prefill``):
    ``S_t = exp(g_t) S_{t-1} + k_t v_t^T``, ``o_t = scale * S_t^T q_t``.

    q, k ``[T, Hk, 128]``, v ``[T, H, 128]`` bf16 (token and head dimensions may be strided; H a
    multiple of Hk); g ``[T, H]`` fp32 log-decays <= 0 (any strides), or ``[H]`` for every token
    alike; cu_seqlens ``[N + 1]`` int32; S_in ``[N, H, 128, 128]`` fp32 or None (zeros).  With
    ``gate`` (``[T, H, 128]`` bf16 logits, may be strided) the output stage is fused:
    ``sigmoid(gate) * norm_weight * o / sqrt(mean(o^2) + eps)``.  S_out may be S_in.
    Returns ``(o, S_out)``: ``[T, H, 128]`` bf16 and ``[N, H, 128, 128]`` fp32.
    """
    good, lib = False, _lib or library()
    try:
        shape, dev = q.shape, q.get_device()
        T, Hk, d = shape
        full = v.shape
        H = full[1]
        qs, ks, vs, gs = q.stride(), k.stride(), v.stride(), g.stride()
        if (dev >= 0 and dev == _here(stream) and dev == k.get_device() == v.get_device() == g.get_device() == cu_seqlens.get_device()
                and q.dtype is k.dtype is v.dtype is _BF16 and g.dtype is _F32 and d == HEAD_DIM and shape == k.shape
                and full == (T, H, d) and g.shape == ((T, H) if len(gs) == 2 else (H,)) and qs[2] == ks[2] == vs[2] == 1 and H % Hk == 0):
            good, gates = _stage_rows(gate, norm_weight, full, dev, _pack3)
            qs, ks, vs, gs = _pack3(*qs), _pack3(*ks), _pack3(*vs), _pack2(*gs) if len(gs) == 2 else _pack2(0, gs[0])
    except (AttributeError, ValueError, TypeError, IndexError, ZeroDivisionError):
        good = False
    if not good:
        (T,), Hk, H, qs, ks, vs, gs, gates = _say_lin_rows(q, k, v, g, gate, norm_weight, 1, "T", _pack2)
        _on(q.get_device(), stream, k, v, g, gate, norm_weight, cu_seqlens if isinstance(cu_seqlens, torch.Tensor) else None)
    n_seq = cu_seqlens.shape[0] - 1 if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dim() == 1 else -1
    if n_seq < 0:
        raise ValueError("cu_seqlens must be a tensor [sequences + 1]")
    states = (n_seq, H, HEAD_DIM, HEAD_DIM)
    cu = _index(cu_seqlens, "cu_seqlens", (n_seq + 1,))
    if S_in is not None:
        _need(S_in, "S_in", _F32, states)
    _on(q.get_device(), stream, S_in, o, S_out, workspace, dev_status)
    if o is None:
        o = _output((T, H, HEAD_DIM), _BF16, q.device, stream)
    else:
        _need(o, "o", _BF16, (T, H, HEAD_DIM))
    S_out = _output(states, _F32, q.device, stream) if S_out is None else _need(S_out, "S_out", _F32, states)
    if workspace is None:
        ws, ws_bytes = None, lib.kda_lin_prefill_workspace_size(n_seq, H, HEAD_DIM, T, n_segments)
        if ws_bytes:
            workspace = _scratch(ws_bytes, q.device, stream)
            ws = workspace.data_ptr()
    else:
        ws, ws_bytes = _workspace(workspace)
    for good in (good, False):
        st = lib.kda_lin_prefill(
            q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, g.data_ptr(), gs, scale, _ptr(gate), gates,
            _ptr(norm_weight), eps, _ptr(S_in), cu, n_seq, T, o.data_ptr(), S_out.data_ptr(), Hk, H, HEAD_DIM, n_segments, ws,
            ws_bytes, _status_ptr(dev_status), _stream_of(stream))
        if st != _ALIGNMENT or not good:
            break
        _, _, _, qs, ks, vs, gs, gates = _say_lin_rows(q, k, v, g, gate, norm_weight, 1, "T", _pack2)
    if st != 0:
        raise KdaError(st, "kda_lin_prefill")
    return o, S_out


def lin_decode(q, k, v, g, S_state, n_commit=None, scale=1.0, gate=None, norm_weight=None, eps=1e-5, o=None,
               dev_status=None, stream=None):
    """:func:`lin_prefill` for a decode (n_tok = 1) or verify (n_tok <= 4) step in fp32
    (``kda_lin_decode``); updates ``S_state`` ``[B, H, 128, 128]`` in place to the state after
    ``n_commit`` ``[B]`` int32 tokens (None: all; 0 leaves it untouched).

    q, k ``[B, n_tok, Hk, 128]``, v and gate ``[B, n_tok, H, 128]`` bf16 (leading dimensions may be
    strided); g ``[B, n_tok, H]`` or ``[H]`` fp32.  Returns o ``[B, n_tok, H, 128]`` fp32.
    """
    good = False
    try:
        shape, dev = q.shape, q.get_device()
        B, n_tok, Hk, d = shape
        full = v.shape
        H = full[2]
        qs, ks, vs, gs = q.stride(), k.stride(), v.stride(), g.stride()
        if (dev >= 0 and dev == _here(stream) and dev == k.get_device() == v.get_device() == g.get_device() == S_state.get_device()
                and q.dtype is k.dtype is v.dtype is _BF16 and g.dtype is _F32 and d == HEAD_DIM and shape == k.shape
                and full == (B, n_tok, H, d) and g.shape == ((B, n_tok, H) if len(gs) == 3 else (H,))
                and qs[3] == ks[3] == vs[3] == 1 and H % Hk == 0):
            good, gates = _stage_rows(gate, norm_weight, full, dev, _pack4)
            qs, ks, vs, gs = _pack4(*qs), _pack4(*ks), _pack4(*vs), _pack3(*gs) if len(gs) == 3 else _pack3(0, 0, gs[0])
    except (AttributeError, ValueError, TypeError, IndexError, ZeroDivisionError):
        good = False
    if not good:
        (B, n_tok), Hk, H, qs, ks, vs, gs, gates = _say_lin_rows(q, k, v, g, gate, norm_weight, 2, "B, n_tok", _pack3)
        _on(q.get_device(), stream, k, v, g, gate, norm_weight)
    _need(S_state, "S_state", _F32, (B, H, HEAD_DIM, HEAD_DIM))
    commit = None if n_commit is None else _index(n_commit, "n_commit", (B,))
    _on(q.get_device(), stream, S_state, n_commit, o, dev_status)
    if o is None:
        o = _output((B, n_tok, H, HEAD_DIM), _F32, q.device, stream)
    else:
        _need(o, "o", _F32, (B, n_tok, H, HEAD_DIM))
    for good in (good, False):
        st = (_lib or library()).kda_lin_decode(
            q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, g.data_ptr(), gs, scale, _ptr(gate), gates,
            _ptr(norm_weight), eps, S_state.data_ptr(), commit, o.data_ptr(), B, n_tok, Hk, H, HEAD_DIM,
            _status_ptr(dev_status), _stream_of(stream))
        if st != _ALIGNMENT or not good:
            break
        _, _, _, qs, ks, vs, gs, gates = _say_lin_rows(q, k, v, g, gate, norm_weight, 2, "B, n_tok", _pack3)
    if st != 0:
        raise KdaError(st, "kda_lin_decode")
    return o


def _wide_rows(t, name, dtypes, shape):
    """Elements from one row to the next of ``t`` ``[rows, width]``; the rows may be strided."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {'[rows, width]' if shape is None else tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.shape[0] and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def block_norm(x, weight=None, y=None, post_norm=False, post_weight=None, gate=None, scale=1.0, eps=1e-5, h=None,
               x_out=None, stream=None):
    """The step between two blocks, in one pass (``kda_block_norm``):
    ``x' = x + scale * sigmoid(gate) * post_weight * N(y)`` and
    ``h = weight * x' / sqrt(mean(x'^2) + eps)``, N the same norm with ``post_norm``, else nothing.

    x ``[T, W]`` the residual stream, bf16 or fp32; y ``[T, W]`` bf16 the block's output, or None (the
    norm in front of the first block); gate ``[T, W]`` bf16 logits or None; weight, post_weight ``[W]``
    fp32 or None (ones).  Rows may be strided; W a multiple of 8.  Returns ``(h, x')``: h ``[T, W]``
    bf16; x' of x's type, in ``x_out`` (contiguous; may be x) when given, and x itself without y.  A row's last bits
    may depend on the number of rows in the call.
    """
    try:
        shape, dev, dtype = x.shape, x.get_device(), x.dtype
        T, W = shape
        xs, one = x.stride()
        ys = gs = 0
        good = (dev >= 0 and dev == _here(stream) and one == 1 and T > 1 and (dtype is _BF16 or dtype is _F32)
                and (weight is None or (weight.shape == (W,) and weight.dtype is _F32 and weight.get_device() == dev and weight.is_contiguous())))
        if good and y is not None:
            ys, one = y.stride()
            good = y.shape == shape and y.dtype is _BF16 and y.get_device() == dev and one == 1
            if post_weight is not None:
                good = (good and post_weight.shape == (W,) and post_weight.dtype is _F32 and post_weight.get_device() == dev
                        and post_weight.is_contiguous())
            if gate is not None:
                gs, one = gate.stride()
                good = good and gate.shape == shape and gate.dtype is _BF16 and gate.get_device() == dev and one == 1
        elif gate is not None or post_norm or post_weight is not None or x_out is not None:
            good = False
    except (AttributeError, ValueError):
        good = False
    if not good:  # say what is wrong, or take what the quick look does not
        xs = _wide_rows(x, "x", (_BF16, _F32), None)
        shape, dtype = x.shape, x.dtype
        T, W = shape
        ys = gs = 0
        if y is not None:
            ys = _wide_rows(y, "y", (_BF16,), shape)
            if gate is not None:
                gs = _wide_rows(gate, "gate", (_BF16,), shape)
            if post_weight is not None:
                _need(post_weight, "post_weight", _F32, (W,))
        elif gate is not None or post_norm or post_weight is not None:
            raise ValueError("post_norm, post_weight and gate belong to a block's output y")
        elif x_out is not None:
            raise ValueError("x_out needs a block's output y")
        if weight is not None:
            _need(weight, "weight", _F32, (W,))
        _on(x.get_device(), stream, y, gate, weight, post_weight)
    if h is not None or x_out is not None:
        _on(x.get_device(), stream, h, x_out)
    if y is not None:
        x_out = _output(shape, dtype, x.device, stream) if x_out is None else _need(x_out, "x_out", dtype, shape)
    h = _output(shape, _BF16, x.device, stream) if h is None else _need(h, "h", _BF16, shape)
    st = (_lib or library()).kda_block_norm(
        x.data_ptr(), 0 if dtype is _BF16 else 1, xs, _ptr(weight), _ptr(y), ys, post_norm, _ptr(post_weight), _ptr(gate),
        gs, scale, eps, h.data_ptr(), _ptr(x_out), T, W, _stream_of(stream))
    if st != 0:
        raise KdaError(st, "kda_block_norm")
    return h, x if x_out is None else x_out
