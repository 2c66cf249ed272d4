"""Python binding of libattn.so: the C entry points under the same names.

Argument marshalling only: every step of the computation runs in the CUDA
library. PyTorch supplies device memory and the current stream. If the
library has not been built, ``load()`` raises -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None
_selftest = None

c_int, c_float, c_size_t, c_void_p = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p

ATTN_OK, ATTN_ERR_ARG, ATTN_ERR_ALIGN, ATTN_ERR_LAUNCH, ATTN_ERR_WORKSPACE, ATTN_ERR_TIMEOUT = 0, -1, -2, -3, -4, -5


class _Kv4Struct(ctypes.Structure):
    """attn_kv4_cache of include/attn.h."""
    _fields_ = [("k_codes", c_void_p), ("k_params", c_void_p), ("v_codes", c_void_p), ("v_params", c_void_p),
                ("n_pages", c_int), ("Hkv", c_int), ("d", c_int), ("d_v", c_int)]


class AttnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"attn error {code}: {msg}")
        self.code = code


def _declare(lib):
    lib.attn_fwd.restype = c_int
    lib.attn_fwd.argtypes = [c_void_p] * 5 + [c_int] * 5 + [c_float, c_int, c_void_p, c_void_p]
    lib.attn_fwd_hdim.restype = c_int
    lib.attn_fwd_hdim.argtypes = [c_void_p] * 5 + [c_int] * 6 + [c_float, c_int, c_void_p, c_void_p]
    lib.attn_fwd_gqa.restype = c_int
    lib.attn_fwd_gqa.argtypes = [c_void_p] * 5 + [c_int] * 7 + [c_float, c_int, c_void_p, c_void_p]
    lib.attn_fwd_ex.restype = c_int
    lib.attn_fwd_ex.argtypes = ([c_void_p] * 5 + [c_int] * 7 + [c_float, c_int, c_int, c_int, c_void_p, c_int,
                                                                  c_void_p, c_void_p, c_void_p])
    lib.attn_bwd_ex_workspace_size.restype = c_size_t
    lib.attn_bwd_ex_workspace_size.argtypes = [c_int] * 9
    lib.attn_bwd_ex.restype = c_int
    lib.attn_bwd_ex.argtypes = ([c_void_p] * 9 + [c_int] * 7 + [c_float, c_int, c_int, c_int, c_void_p, c_int,
                                                                  c_void_p, c_void_p, c_int, c_void_p, c_size_t,
                                                                  c_void_p])
    lib.attn_fwd_sinks.restype = c_int
    lib.attn_fwd_sinks.argtypes = ([c_void_p] * 5 + [c_int] * 7 + [c_float, c_int, c_int, c_int, c_int, c_void_p,
                                                                     c_void_p, c_void_p])
    lib.attn_bwd_sinks_workspace_size.restype = c_size_t
    lib.attn_bwd_sinks_workspace_size.argtypes = [c_int] * 12
    lib.attn_bwd_packed_workspace_size.restype = c_size_t
    lib.attn_bwd_packed_workspace_size.argtypes = [c_int] * 12
    lib.attn_bwd_sinks.restype = c_int
    lib.attn_bwd_sinks.argtypes = ([c_void_p] * 9 + [c_int] * 7 + [c_float, c_int, c_int, c_int, c_int, c_void_p,
                                                                     c_void_p, c_int, c_void_p, c_size_t, c_void_p])
    lib.attn_fwd_varlen.restype = c_int
    lib.attn_fwd_varlen.argtypes = [c_void_p] * 5 + [c_int] * 7 + [c_float, c_int, c_void_p, c_void_p, c_void_p]
    lib.attn_bwd_workspace_size.restype = c_size_t
    lib.attn_bwd_workspace_size.argtypes = [c_int] * 7
    lib.attn_bwd.restype = c_int
    lib.attn_bwd.argtypes = ([c_void_p] * 9 + [c_int] * 5 + [c_float, c_int, c_void_p, c_int, c_void_p, c_size_t,
                                                               c_void_p])
    lib.attn_bwd_gqa_workspace_size.restype = c_size_t
    lib.attn_bwd_gqa_workspace_size.argtypes = [c_int] * 8
    lib.attn_bwd_gqa.restype = c_int
    lib.attn_bwd_gqa.argtypes = ([c_void_p] * 9 + [c_int] * 6 + [c_float, c_int, c_void_p, c_int, c_void_p,
                                                                   c_size_t, c_void_p])
    lib.attn_bwd_varlen.restype = c_int
    lib.attn_bwd_varlen.argtypes = ([c_void_p] * 9 + [c_int] * 6 + [c_float, c_int, c_void_p, c_void_p, c_int,
                                                                      c_void_p, c_size_t, c_void_p])
    lib.attn_bwd_noalloc.restype = c_int
    lib.attn_bwd_noalloc.argtypes = [c_void_p] * 9 + [c_int] * 5 + [c_float, c_int, c_void_p, c_int, c_void_p]
    kv4, i64 = ctypes.POINTER(_Kv4Struct), ctypes.c_longlong
    lib.attn_kv4_append.restype = c_int
    lib.attn_kv4_append.argtypes = [c_void_p, c_void_p, i64, i64, kv4, c_void_p, c_int, c_void_p, c_void_p, c_int,
                                    c_int, c_void_p]
    lib.attn_kv4_read.restype = c_int
    lib.attn_kv4_read.argtypes = [c_void_p, c_void_p, kv4, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_void_p]
    lib.attn_kv4_fwd_workspace_size.restype = c_size_t
    lib.attn_kv4_fwd_workspace_size.argtypes = [c_int] * 9
    lib.attn_kv4_fwd.restype = c_int
    lib.attn_kv4_fwd.argtypes = ([c_void_p, i64, kv4, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p]
                                 + [c_int] * 3 + [c_float] + [c_int] * 4
                                 + [c_void_p, i64, c_float, c_void_p, c_size_t, c_void_p])
    lib.attn_kv4_evict.restype = c_int
    lib.attn_kv4_evict.argtypes = ([kv4, c_void_p, c_int, c_void_p, c_void_p, i64, c_void_p] + [c_int] * 5
                                   + [c_void_p] * 3 + [i64, c_void_p])
    lib.attn_set_backward_cta_pairs.restype = c_int
    lib.attn_set_backward_cta_pairs.argtypes = [c_int]
    lib.attn_set_exp2_emulation.restype = c_int
    lib.attn_set_exp2_emulation.argtypes = [c_int, c_int]
    lib.attn_last_error.restype = ctypes.c_char_p
    lib.attn_last_error.argtypes = []
    lib.attn_check_status.restype = c_int
    lib.attn_check_status.argtypes = [c_void_p]
    lib.attn_version.restype = c_int
    lib.attn_version.argtypes = []
    return lib


def library_path() -> str:
    return _build.lib_path("libattn.so")


def load():
    """Load libattn.so (built by ``build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: run exact_attention_blackwell_tma_gb300.build.build() "
                                   "(or __graft_entry__.build()) first; there is no CPU fallback")
            _lib = _declare(ctypes.CDLL(path))
    return _lib


def load_selftest():
    global _selftest
    with _lock:
        if _selftest is None:
            path = _build.lib_path("libattn_selftest.so")
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build first")
            lib = ctypes.CDLL(path)
            lib.attn_selftest_mma.restype = c_int
            lib.attn_selftest_mma.argtypes = [c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
            lib.attn_selftest_exp2.restype = c_int
            lib.attn_selftest_exp2.argtypes = [c_void_p, c_void_p, c_void_p, c_int, c_void_p]
            lib.attn_selftest_wait_timeout.restype = c_int
            lib.attn_selftest_wait_timeout.argtypes = [c_void_p, ctypes.c_ulonglong, c_void_p]
            _selftest = lib
    return _selftest


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without building the Stream object (3 us); torch does not promise this name
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        return (torch.cuda.current_stream().cuda_stream if _raw_stream is None
                else _raw_stream(torch.cuda.current_device()))
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def last_error() -> str:
    return load().attn_last_error().decode()


def _check(rc: int):
    if rc != ATTN_OK:
        raise AttnError(rc, last_error())


# ---------------------------------------------------------------- C entry points, same names

def attn_fwd(q, k, v, o, lse, B, H, Lq, Lk, d, scale, causal, cu_seqlens=None, stream=None) -> int:
    return load().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, scale, int(causal),
                           _ptr(cu_seqlens), _stream(stream))

def attn_fwd_hdim(q, k, v, o, lse, B, H, Lq, Lk, d, dv, scale, causal, cu_seqlens=None, stream=None) -> int:
    return load().attn_fwd_hdim(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, dv, scale,
                                int(causal), _ptr(cu_seqlens), _stream(stream))


def attn_fwd_gqa(q, k, v, o, lse, B, H, Hkv, Lq, Lk, d, dv, scale, causal, cu_seqlens=None, stream=None) -> int:
    return load().attn_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Lq, Lk, d, dv, scale,
                               int(causal), _ptr(cu_seqlens), _stream(stream))


def attn_fwd_varlen(q, k, v, o, lse, B, H, Hkv, Tq, Tk, d, dv, scale, causal, cu_seqlens_q, cu_seqlens_k,
                    stream=None) -> int:
    return load().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Tq, Tk, d, dv, scale,
                                  int(causal), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _stream(stream))


def attn_fwd_ex(q, k, v, o, lse, B, H, Hkv, Lq, Lk, d, d_v, scale, causal, window_left=-1, window_right=-1,
                block_mask=None, mask_heads=1, cu_seqlens_q=None, cu_seqlens_k=None, stream=None) -> int:
    return load().attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Lq, Lk, d, d_v, scale,
                              int(causal), int(window_left), int(window_right), _ptr(block_mask), int(mask_heads),
                              _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _stream(stream))


def attn_bwd_ex_workspace_size(B, H, Hkv, Lq, Lk, d, d_v, causal, deterministic) -> int:
    return load().attn_bwd_ex_workspace_size(B, H, Hkv, Lq, Lk, d, d_v, int(causal), int(deterministic))


def attn_bwd_ex(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Lq, Lk, d, d_v, scale, causal, window_left,
                window_right, block_mask, mask_heads, cu_seqlens_q, cu_seqlens_k, deterministic, workspace, ws_bytes,
                stream=None) -> int:
    return load().attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                              _ptr(dv), B, H, Hkv, Lq, Lk, d, d_v, scale, int(causal), int(window_left),
                              int(window_right), _ptr(block_mask), int(mask_heads), _ptr(cu_seqlens_q),
                              _ptr(cu_seqlens_k), int(deterministic), _ptr(workspace), ws_bytes, _stream(stream))


def attn_fwd_sinks(q, k, v, o, lse, B, H, Hkv, Lq, Lk, d, d_v, scale, causal, window_left, window_right, sinks,
                   cu_seqlens_q=None, cu_seqlens_k=None, stream=None) -> int:
    return load().attn_fwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Lq, Lk, d, d_v, scale,
                                 int(causal), int(window_left), int(window_right), int(sinks), _ptr(cu_seqlens_q),
                                 _ptr(cu_seqlens_k), _stream(stream))


def attn_bwd_sinks_workspace_size(B, H, Hkv, Lq, Lk, d, d_v, causal, window_left, window_right, sinks,
                                  deterministic) -> int:
    return load().attn_bwd_sinks_workspace_size(B, H, Hkv, Lq, Lk, d, d_v, int(causal), int(window_left),
                                                int(window_right), int(sinks), int(deterministic))


def attn_bwd_packed_workspace_size(B, H, Hkv, Tq, Tk, d, d_v, causal, window_left, window_right, sinks,
                                   deterministic) -> int:
    return load().attn_bwd_packed_workspace_size(B, H, Hkv, Tq, Tk, d, d_v, int(causal), int(window_left),
                                                 int(window_right), int(sinks), int(deterministic))


def attn_bwd_sinks(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Lq, Lk, d, d_v, scale, causal, window_left,
                   window_right, sinks, cu_seqlens_q, cu_seqlens_k, deterministic, workspace, ws_bytes,
                   stream=None) -> int:
    return load().attn_bwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                 _ptr(dv), B, H, Hkv, Lq, Lk, d, d_v, scale, int(causal), int(window_left),
                                 int(window_right), int(sinks), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                 int(deterministic), _ptr(workspace), ws_bytes, _stream(stream))


def attn_bwd_workspace_size(B, H, Lq, Lk, d, causal, deterministic) -> int:
    return load().attn_bwd_workspace_size(B, H, Lq, Lk, d, int(causal), int(deterministic))


def attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, Lq, Lk, d, scale, causal, cu_seqlens, deterministic,
             workspace, ws_bytes, stream=None) -> int:
    return load().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                           _ptr(dv), B, H, Lq, Lk, d, scale, int(causal), _ptr(cu_seqlens), int(deterministic),
                           _ptr(workspace), ws_bytes, _stream(stream))


def attn_bwd_gqa_workspace_size(B, H, Hkv, Lq, Lk, d, causal, deterministic) -> int:
    return load().attn_bwd_gqa_workspace_size(B, H, Hkv, Lq, Lk, d, int(causal), int(deterministic))


def attn_bwd_gqa(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Lq, Lk, d, scale, causal, cu_seqlens, deterministic,
                 workspace, ws_bytes, stream=None) -> int:
    return load().attn_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                               _ptr(dv), B, H, Hkv, Lq, Lk, d, scale, int(causal), _ptr(cu_seqlens),
                               int(deterministic), _ptr(workspace), ws_bytes, _stream(stream))


def attn_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Tq, Tk, d, scale, causal, cu_seqlens_q,
                    cu_seqlens_k, deterministic, workspace, ws_bytes, stream=None) -> int:
    return load().attn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                  _ptr(dv), B, H, Hkv, Tq, Tk, d, scale, int(causal), _ptr(cu_seqlens_q),
                                  _ptr(cu_seqlens_k), int(deterministic), _ptr(workspace), ws_bytes,
                                  _stream(stream))


def attn_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H, Lq, Lk, d, scale, causal, cu_seqlens,
                     deterministic, stream=None) -> int:
    """attn_bwd without a workspace: scratch comes from a fixed array inside the
    library (for callers that cannot allocate device memory; see include/attn.h)."""
    return load().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                                   _ptr(dk), _ptr(dv), B, H, Lq, Lk, d, scale, int(causal), _ptr(cu_seqlens),
                                   int(deterministic), _stream(stream))


def attn_kv4_append(k, v, k_stride, v_stride, cache, page_table, table_width, cache_lens, cu_seqlens, B, L,
                    stream=None) -> int:
    return load().attn_kv4_append(_ptr(k), _ptr(v), k_stride, v_stride, cache, _ptr(page_table), table_width,
                                  _ptr(cache_lens), _ptr(cu_seqlens), B, L, _stream(stream))


def attn_kv4_read(k, v, cache, page_table, table_width, cache_lens, cu_seqlens, B, L, stream=None) -> int:
    return load().attn_kv4_read(_ptr(k), _ptr(v), cache, _ptr(page_table), table_width, _ptr(cache_lens),
                                _ptr(cu_seqlens), B, L, _stream(stream))


def attn_kv4_fwd_workspace_size(B, H, Hkv, L, packed, table_width, d, d_v, key_weights) -> int:
    return load().attn_kv4_fwd_workspace_size(B, H, Hkv, L, int(packed), table_width, d, d_v, int(key_weights))


def attn_kv4_fwd(q, q_stride, cache, page_table, table_width, cache_lens, cu_seqlens, o, lse, B, H, L, scale, causal,
                 window_left, window_right, sinks, key_weights, weight_stride, weight_decay, workspace, ws_bytes,
                 stream=None) -> int:
    return load().attn_kv4_fwd(_ptr(q), q_stride, cache, _ptr(page_table), table_width, _ptr(cache_lens),
                               _ptr(cu_seqlens), _ptr(o), _ptr(lse), B, H, L, scale, int(causal), int(window_left),
                               int(window_right), int(sinks), _ptr(key_weights), weight_stride, weight_decay,
                               _ptr(workspace), ws_bytes, _stream(stream))


def attn_kv4_evict(cache, page_table, table_width, cache_lens, key_weights, weight_stride, new_table, new_width, B,
                   budget, sinks, recent, new_lens, kept, new_key_weights, new_weight_stride, stream=None) -> int:
    return load().attn_kv4_evict(cache, _ptr(page_table), table_width, _ptr(cache_lens), _ptr(key_weights),
                                 weight_stride, _ptr(new_table), new_width, B, budget, sinks, recent, _ptr(new_lens),
                                 _ptr(kept), _ptr(new_key_weights), new_weight_stride, _stream(stream))


def attn_set_backward_cta_pairs(enable) -> int:
    """Backward main kernel on CTA pairs (2-CTA tensor cores) where it applies;
    returns the previous setting."""
    return load().attn_set_backward_cta_pairs(int(bool(enable)))


def attn_set_exp2_emulation(d, every) -> int:
    """Forward exp2 emulation for head dim d: one column pair in `every` (0, 4, 8)
    by the FMA polynomial; returns the previous setting (or a negative code)."""
    return load().attn_set_exp2_emulation(int(d), int(every))


def attn_last_error() -> str:
    return last_error()


def attn_check_status(stream=None) -> int:
    return load().attn_check_status(_stream(stream))


# ---------------------------------------------------------------- tensor-level helpers

def _dims(q, k, cu_seqlens):
    """B, H, Lq, Lk, d and the key/value heads Hkv."""
    if cu_seqlens is None:
        B, Lq, H, d = q.shape
        return B, H, Lq, k.shape[1], d, k.shape[2]
    T, H, d = q.shape
    return cu_seqlens.numel() - 1, H, T, k.shape[0], d, k.shape[1]


def _mask_heads(block_mask, H, Lq, Lk):
    """Heads of a block mask after checking its shape [Hm, ceil(Lq/128), ceil(Lk/128)] (2-D: Hm = 1)."""
    if block_mask is None:
        return 1
    shape = tuple(block_mask.shape)
    want = (-(-Lq // 128), -(-Lk // 128))
    if block_mask.dtype != torch.uint8 or not (shape == want or (len(shape) == 3 and shape[1:] == want
                                                                 and shape[0] in (1, H))):
        raise ValueError(f"block_mask must be uint8 [1 or {H}, {want[0]}, {want[1]}], got {block_mask.dtype} {shape}")
    return 1 if len(shape) == 2 else shape[0]


# functions of the sizes alone
_sinks_workspace = functools.lru_cache(maxsize=4096)(attn_bwd_sinks_workspace_size)
_packed_workspace = functools.lru_cache(maxsize=4096)(attn_bwd_packed_workspace_size)


def _no_block_mask(block_mask):
    if block_mask is not None:
        raise ValueError("sinks are not combined with a block mask")


def _check_tensors(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def _check_ints(*bounds):
    """Window bounds, sinks and budgets: ctypes keeps the low 32 bits of an integer without a word."""
    for x in bounds:
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{x} (of {bounds}) does not fit an int")


def _check_workspace(workspace, device):
    """A caller's workspace goes to the kernels as it is: it has to lie on their device (an index)."""
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on cuda:{device}, got one on {workspace.device}")


def forward(q, k, v, causal: bool, scale: float | None = None, cu_seqlens=None, out=None, lse=None,
            stream=None, cu_seqlens_k=None, window=(-1, -1), block_mask=None, sinks=0):
    """O, LSE for bf16 q, k, v ([B, L, H, d], or [T, H, d] with int32 cu_seqlens).
    v (and O) may have a head dim of their own (d = 192 with 128); k and v may
    have fewer heads than q (grouped heads: query head h reads h // (H // Hkv)).
    cu_seqlens_k: key offsets of a varlen batch whose key lengths differ.
    window: (left, right) bounds of a local window, -1 for an open side.
    sinks: the first keys of each sequence that stay visible left of the window
    (not with a block mask).
    block_mask: uint8 CUDA tensor [Hm, ceil(Lq/128), ceil(Lk/128)] (Hm 1 or H;
    2-D means Hm = 1), dense problems only; zero drops a 128 x 128 block."""
    _check_tensors(q, k, v, cu_seqlens, cu_seqlens_k)
    B, H, Lq, Lk, d, Hkv = _dims(q, k, cu_seqlens)
    dv = v.shape[-1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty(q.shape[:-1] + (dv,), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Lq) if cu_seqlens is None else (H, Lq), dtype=torch.float32, device=q.device)
    if sinks:
        _no_block_mask(block_mask)
        _check_ints(window[0], window[1], sinks)
        _check(load().attn_fwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv,
                                     Lq, Lk, d, dv, scale, int(causal), window[0], window[1], sinks, _ptr(cu_seqlens),
                                     _ptr(cu_seqlens_k), _stream(stream)))
    elif tuple(window) != (-1, -1) or block_mask is not None:
        mh = _mask_heads(block_mask, H, Lq, Lk)
        _check_tensors(block_mask)
        _check(attn_fwd_ex(q, k, v, out, lse, B, H, Hkv, Lq, Lk, d, dv, scale, causal, window[0], window[1],
                           block_mask, mh, cu_seqlens, cu_seqlens_k, stream))
    elif cu_seqlens_k is not None:
        _check(attn_fwd_varlen(q, k, v, out, lse, B, H, Hkv, Lq, Lk, d, dv, scale, causal, cu_seqlens,
                               cu_seqlens_k, stream))
    elif Hkv != H:
        _check(attn_fwd_gqa(q, k, v, out, lse, B, H, Hkv, Lq, Lk, d, dv, scale, causal, cu_seqlens, stream))
    elif dv == d:
        _check(attn_fwd(q, k, v, out, lse, B, H, Lq, Lk, d, scale, causal, cu_seqlens, stream))
    else:
        _check(attn_fwd_hdim(q, k, v, out, lse, B, H, Lq, Lk, d, dv, scale, causal, cu_seqlens, stream))
    return out, lse


def backward(q, k, v, o, lse, dout, causal: bool, scale: float | None = None, cu_seqlens=None,
             deterministic: bool = False, workspace=None, dq=None, dk=None, dv=None, stream=None,
             cu_seqlens_k=None, window=(-1, -1), block_mask=None, sinks=0):
    """dQ, dK, dV (bf16) for the loss sum(O * dO); k and v may have fewer heads
    than q (grouped heads), dK and dV then have theirs; v (dO, dV) may have a head
    dim of its own (d = 192 with 128). cu_seqlens_k, window, block_mask and sinks as in forward()."""
    _check_tensors(q, k, v, o, lse, dout, cu_seqlens, cu_seqlens_k)
    B, H, Lq, Lk, d, Hkv = _dims(q, k, cu_seqlens)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    d_v = v.shape[-1]
    if sinks:
        _check_ints(window[0], window[1], sinks)
    if cu_seqlens is not None:
        need = _packed_workspace(B, H, Hkv, Lq, Lk, d, d_v, causal, window[0], window[1], sinks, deterministic)
    elif sinks:
        need = _sinks_workspace(B, H, Hkv, Lq, Lk, d, d_v, causal, window[0], window[1], sinks, deterministic)
    else:
        need = attn_bwd_ex_workspace_size(B, H, Hkv, Lq, Lk, d, d_v, causal, deterministic)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    else:
        _check_workspace(workspace, q.get_device())
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws_bytes = workspace.numel() * workspace.element_size()
    if sinks:
        _no_block_mask(block_mask)
        _check(load().attn_bwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                     dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Hkv, Lq, Lk, d,
                                     d_v, scale, int(causal), window[0], window[1], sinks, _ptr(cu_seqlens),
                                     _ptr(cu_seqlens_k), int(deterministic), workspace.data_ptr(), ws_bytes,
                                     _stream(stream)))
    elif d_v != d or tuple(window) != (-1, -1) or block_mask is not None:
        mh = _mask_heads(block_mask, H, Lq, Lk)
        _check_tensors(block_mask)
        _check(attn_bwd_ex(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Lq, Lk, d, d_v, scale, causal, window[0],
                           window[1], block_mask, mh, cu_seqlens, cu_seqlens_k, deterministic, workspace, ws_bytes,
                           stream))
    elif cu_seqlens_k is not None:
        _check(attn_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Lq, Lk, d, scale, causal, cu_seqlens,
                               cu_seqlens_k, deterministic, workspace, ws_bytes, stream))
    elif Hkv != H:
        _check(attn_bwd_gqa(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, Lq, Lk, d, scale, causal, cu_seqlens,
                            deterministic, workspace, ws_bytes, stream))
    else:
        _check(attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, Lq, Lk, d, scale, causal, cu_seqlens,
                        deterministic, workspace, ws_bytes, stream))
    return dq, dk, dv


def check_status(stream=None):
    _check(attn_check_status(stream))


# ---------------------------------------------------------------- the 4-bit key/value cache

KV4_PAGE, KV4_GROUP = 64, 64   # tokens of a page; channels that share a scale and a minimum


class Kv4Cache:
    """The four tensors of a 4-bit cache (layout: include/attn.h, attn_kv4_cache):
    k_codes uint8 [pages, Hkv, d // 64, 64, 32], k_params bf16 [pages, Hkv, d // 64, 64, 2],
    v_codes and v_params the same with v's head dim."""

    __slots__ = ("k_codes", "k_params", "v_codes", "v_params", "n_pages", "Hkv", "d", "dv", "device", "_struct")

    def __init__(self, k_codes, k_params, v_codes, v_params):
        pages, heads, groups = k_codes.shape[:3]
        v_groups = v_codes.shape[2] if v_codes.dim() == 5 else 0
        rows, dtype, device = (KV4_PAGE, KV4_GROUP // 2), (torch.uint8, torch.bfloat16), k_codes.get_device()
        for codes, params, g in ((k_codes, k_params, groups), (v_codes, v_params, v_groups)):
            if (codes.shape != (pages, heads, g) + rows or params.shape != (pages, heads, g, KV4_PAGE, 2)
                    or (codes.dtype, params.dtype) != dtype or codes.get_device() != device
                    or params.get_device() != device):
                raise ValueError(f"a 4-bit cache needs uint8 codes [pages, heads, groups, {KV4_PAGE}, {KV4_GROUP // 2}] "
                                 f"and bf16 params [pages, heads, groups, {KV4_PAGE}, 2] on one device, got {codes.dtype} "
                                 f"{tuple(codes.shape)} and {params.dtype} {tuple(params.shape)}")
        _check_tensors(k_codes, k_params, v_codes, v_params)
        self.k_codes, self.k_params, self.v_codes, self.v_params = k_codes, k_params, v_codes, v_params
        self.n_pages, self.Hkv, self.d, self.dv = pages, heads, groups * KV4_GROUP, v_groups * KV4_GROUP
        self.device = device   # its index
        self._struct = _Kv4Struct(k_codes.data_ptr(), k_params.data_ptr(), v_codes.data_ptr(), v_params.data_ptr(),
                                  self.n_pages, self.Hkv, self.d, self.dv)

    @classmethod
    def empty(cls, n_pages, Hkv, d, dv=None, device="cuda"):
        """A cache of n_pages zeroed pages."""
        dv = d if dv is None else dv
        if d % KV4_GROUP or dv % KV4_GROUP:
            raise ValueError(f"head dims {d}, {dv} of a 4-bit cache must be multiples of {KV4_GROUP}")

        def codes(width):
            return torch.zeros((n_pages, Hkv, width // KV4_GROUP, KV4_PAGE, KV4_GROUP // 2), dtype=torch.uint8,
                               device=device)

        def params(width):
            return torch.zeros((n_pages, Hkv, width // KV4_GROUP, KV4_PAGE, 2), dtype=torch.bfloat16, device=device)
        return cls(codes(d), params(d), codes(dv), params(dv))


def _kv4_int(name, t, dims, rows, device):
    if t.dtype != torch.int32 or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on cuda:{device}")
    shape = t.shape
    if len(shape) != dims or shape[0] != rows:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {dims} dimensions of {rows} rows")


def _kv4_ints(cache, page_table, cache_lens, cu_seqlens, new_table=None):
    """Checks the int32 tensors of a call, which live on the cache's device, the current one; returns (B, device index)."""
    device = cache.device
    if device != torch.cuda.current_device():
        raise ValueError(f"the cache is on cuda:{device}, the current device is cuda:{torch.cuda.current_device()}")
    B = len(cache_lens)
    _kv4_int("cache_lens", cache_lens, 1, B, device)
    _kv4_int("page_table", page_table, 2, B, device)
    if cu_seqlens is not None:
        _kv4_int("cu_seqlens", cu_seqlens, 1, B + 1, device)
    if new_table is not None:
        _kv4_int("new_table", new_table, 2, B, device)
    return B, device


def _kv4_rows(x, heads, width, B, packed, name, device):
    """Rows of [T, heads, width] (packed) or [B, L, heads, width] (dense): (L, elements between rows).
    Heads and channels are contiguous; rows may lie further apart (a slice of a fused projection)."""
    shape, stride = x.shape, x.stride()
    if (len(shape) != (3 if packed else 4) or shape[-2] != heads or shape[-1] != width or x.dtype != torch.bfloat16
            or x.get_device() != device or (not packed and shape[0] != B)):
        lead = "T" if packed else f"{B}, L"
        raise ValueError(f"{name} must be a bf16 tensor [{lead}, {heads}, {width}] on cuda:{device}, got {x.dtype} "
                         f"{tuple(shape)} on {x.device}")
    L = shape[-3]
    if L == 0 or (not packed and B == 0):
        return L, heads * width
    row = stride[-3] if L > 1 else (stride[0] if not packed and B > 1 else heads * width)
    if stride[-1] != 1 or (heads > 1 and stride[-2] != width) or (not packed and B > 1 and stride[0] != L * row):
        raise ValueError(f"{name}: heads and channels must be contiguous and rows evenly spaced, strides {stride}")
    return L, row


def _kv4_weights(key_weights, B, cache, device):
    if (key_weights.dtype != torch.float32 or key_weights.get_device() != device or not key_weights.is_contiguous()
            or key_weights.dim() != 3 or key_weights.shape[0] != B or key_weights.shape[1] != cache.Hkv):
        raise ValueError(f"key_weights must be a contiguous fp32 tensor [{B}, {cache.Hkv}, keys] on cuda:{device}")


def _kv4_out(t, shape, dtype, device, name):
    """An output tensor: the caller's, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {device}")
    return t


_kv4_workspace = functools.lru_cache(maxsize=4096)(attn_kv4_fwd_workspace_size)   # a function of the sizes alone


def _on(stream):
    """Allocations inside belong to the stream that the call runs on."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def kv4_append(cache, k, v, page_table, cache_lens, cu_seqlens=None, stream=None):
    """Quantise new keys and values (bf16 [T, Hkv, d] with int32 cu_seqlens, or [B, L, Hkv, d]) into the pages of
    their sequences. cache_lens (int32 [B]) counts the new tokens already: sequence b's n rows become its tokens
    cache_lens[b] - n .. cache_lens[b] - 1. Rows of k and v may be strided (a slice of a fused projection)."""
    B, device = _kv4_ints(cache, page_table, cache_lens, cu_seqlens)
    L, k_stride = _kv4_rows(k, cache.Hkv, cache.d, B, cu_seqlens is not None, "k", device)
    Lv, v_stride = _kv4_rows(v, cache.Hkv, cache.dv, B, cu_seqlens is not None, "v", device)
    if L != Lv:
        raise ValueError(f"k has {L} rows, v {Lv}")
    _check(load().attn_kv4_append(k.data_ptr(), v.data_ptr(), k_stride, v_stride, cache._struct, page_table.data_ptr(),
                                  page_table.shape[1], cache_lens.data_ptr(), _ptr(cu_seqlens), B, L, _stream(stream)))


def kv4_read(cache, page_table, cache_lens, rows, cu_seqlens=None, k=None, v=None, stream=None):
    """K, V in bf16 as the cache stands for them: the last rows of every sequence, packed ([rows, Hkv, d], rows =
    cu_seqlens[-1]) or dense (rows per sequence; [B, rows, Hkv, d], zero before a sequence's first token)."""
    B, _ = _kv4_ints(cache, page_table, cache_lens, cu_seqlens)
    device, heads = cache.k_codes.device, cache.Hkv
    packed = cu_seqlens is not None
    with _on(stream):
        k = _kv4_out(k, (rows, heads, cache.d) if packed else (B, rows, heads, cache.d), torch.bfloat16, device, "k")
        v = _kv4_out(v, (rows, heads, cache.dv) if packed else (B, rows, heads, cache.dv), torch.bfloat16, device, "v")
    _check(load().attn_kv4_read(k.data_ptr(), v.data_ptr(), cache._struct, page_table.data_ptr(), page_table.shape[1],
                                cache_lens.data_ptr(), _ptr(cu_seqlens), B, rows, _stream(stream)))
    return k, v


def kv4_forward(q, cache, page_table, cache_lens, causal: bool = True, scale: float | None = None, cu_seqlens=None,
                window=(-1, -1), sinks: int = 0, key_weights=None, weight_decay: float = 1.0, out=None, lse=None,
                workspace=None, stream=None):
    """O, LSE of new tokens q (bf16 [T, H, d] with cu_seqlens, or [B, L, H, d]) over their sequence's cache, to which
    their keys have been appended. window and sinks as in forward(). key_weights (fp32 [B, Hkv, >= longest cache]):
    updated in place to weight_decay * key_weights + the attention weight each key got from the call's rows."""
    B, index = _kv4_ints(cache, page_table, cache_lens, cu_seqlens)
    _check_ints(window[0], window[1], sinks)
    H, packed, device = q.shape[-2], cu_seqlens is not None, q.device
    L, q_stride = _kv4_rows(q, H, cache.d, B, packed, "q", index)
    if H % cache.Hkv != 0 or H == 0:
        raise ValueError(f"{H} query heads over {cache.Hkv} key/value heads")
    if key_weights is not None:
        _kv4_weights(key_weights, B, cache, index)
    scale = 1.0 / math.sqrt(cache.d) if scale is None else scale
    width = page_table.shape[1]
    need = _kv4_workspace(B, H, cache.Hkv, L, packed, width, cache.d, cache.dv, key_weights is not None)
    with _on(stream):
        out = _kv4_out(out, (L, H, cache.dv) if packed else (B, L, H, cache.dv), torch.bfloat16, device, "out")
        lse = _kv4_out(lse, (H, L) if packed else (B, H, L), torch.float32, device, "lse")
        if workspace is None:
            workspace, size = torch.empty(max(need, 1), dtype=torch.uint8, device=device), need
        else:
            _check_workspace(workspace, index)
            size = workspace.numel() * workspace.element_size()
    _check(load().attn_kv4_fwd(q.data_ptr(), q_stride, cache._struct, page_table.data_ptr(), width, cache_lens.data_ptr(),
                               _ptr(cu_seqlens), out.data_ptr(), lse.data_ptr(), B, H, L, scale, int(causal),
                               window[0], window[1], sinks, _ptr(key_weights),
                               0 if key_weights is None else key_weights.shape[2], weight_decay, workspace.data_ptr(),
                               size, _stream(stream)))
    return out, lse


def kv4_evict(cache, page_table, cache_lens, key_weights, new_table, budget: int, sinks: int = 0, recent: int = 0,
              new_lens=None, kept=None, new_key_weights=None, stream=None):
    """Keep, of every sequence longer than budget and for each key/value head, the first `sinks` keys, the last
    `recent` and those between with the largest key_weights, in the pages of new_table (pages of the same cache that
    are not in page_table). Returns new_lens int32 [B], kept int32 [B, Hkv, budget] (old token of each new one, -1 past
    the new length) and the kept key weights fp32 [B, Hkv, budget] (or as wide as new_key_weights is)."""
    B, index = _kv4_ints(cache, page_table, cache_lens, None, new_table)
    _kv4_weights(key_weights, B, cache, index)
    _check_ints(budget, sinks, recent)
    device = cache_lens.device
    columns = budget if new_key_weights is None else new_key_weights.shape[-1]
    with _on(stream):
        new_lens = _kv4_out(new_lens, (B,), torch.int32, device, "new_lens")
        kept = _kv4_out(kept, (B, cache.Hkv, budget), torch.int32, device, "kept")
        new_key_weights = _kv4_out(new_key_weights, (B, cache.Hkv, columns), torch.float32, device, "new_key_weights")
    _check(load().attn_kv4_evict(cache._struct, page_table.data_ptr(), page_table.shape[1], cache_lens.data_ptr(),
                                 key_weights.data_ptr(), key_weights.shape[2], new_table.data_ptr(), new_table.shape[1],
                                 B, budget, sinks, recent, new_lens.data_ptr(), kept.data_ptr(),
                                 new_key_weights.data_ptr(), columns, _stream(stream)))
    return new_lens, kept, new_key_weights
