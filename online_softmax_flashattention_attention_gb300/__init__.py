"""Python binding of the fused attention forward library (``libattn.so``, C ABI in include/attn.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and streams.  There
is no fallback: if the library is missing or a call fails, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
import weakref

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn.so")

EXPORTS = ("attn_fwd", "attn_fwd_ex", "attn_fwd_strided", "attn_fwd_varlen", "attn_fwd_host", "attn_release_workspace", "attn_status_sync", "attn_last_error",
           "attn_version", "attn_fwd_noalloc", "attn_fwd_states", "attn_merge_states",
           "attn_splitkv_workspace_bytes", "attn_splitkv_splits", "attn_fwd_splitkv",
           "attn_cache_write", "attn_cache_read", "attn_cache_check", "attn_fwd_tree", "attn_tree_workspace_bytes",
           "attn_qk_rotate", "attn_fwd_prompt", "attn_prompt_workspace_bytes", "attn_cache_weigh", "attn_cache_evict")

STATUS_NAMES = {0: "ATTN_OK", -1: "ATTN_ERR_NULLPTR", -2: "ATTN_ERR_BAD_SHAPE", -3: "ATTN_ERR_UNSUPPORTED_D",
                -4: "ATTN_ERR_MISALIGNED", -5: "ATTN_ERR_NO_DEVICE", -6: "ATTN_ERR_LAUNCH", -7: "ATTN_ERR_TIMEOUT",
                -8: "ATTN_ERR_BAD_ARG", -9: "ATTN_ERR_BAD_PAGE"}


EXP2_DEFAULT, EXP2_HARDWARE, EXP2_MIXED = 0, 1, 2


class AttnOptions(ctypes.Structure):
    """attn_options of include/attn.h."""
    _fields_ = [("size", ctypes.c_size_t), ("rescale_threshold", ctypes.c_float), ("exp2_mode", ctypes.c_int),
                ("key_block", ctypes.c_int)]


CACHE_BF16, CACHE_E4M3 = 0, 1


class AttnCache(ctypes.Structure):
    """attn_cache of include/attn.h."""
    _fields_ = [("size", ctypes.c_size_t), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("type", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("num_heads", ctypes.c_int),
                ("d", ctypes.c_int)]


class AttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def load_library():
    """Load libattn.so (built by ``__graft_entry__.build()``); raises if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        sig = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp]
        for name in ("attn_fwd", "attn_fwd_host"):
            getattr(lib, name).argtypes = sig
            getattr(lib, name).restype = i
        lib.attn_release_workspace.argtypes = []
        lib.attn_release_workspace.restype = i
        lib.attn_status_sync.argtypes = [vp]
        lib.attn_status_sync.restype = i
        lib.attn_last_error.argtypes = []
        lib.attn_last_error.restype = ctypes.c_char_p
        lib.attn_version.argtypes = []
        lib.attn_version.restype = i
        lib.attn_fwd_ex.argtypes = sig[:-1] + [ctypes.POINTER(AttnOptions), vp]
        lib.attn_fwd_ex.restype = i
        i64p = ctypes.POINTER(ctypes.c_int64)
        lib.attn_fwd_strided.argtypes = sig[:-1] + [i64p, i64p, i64p, i64p, vp]
        lib.attn_fwd_strided.restype = i
        lib.attn_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        lib.attn_fwd_varlen.restype = i
        lib.attn_fwd_states.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, vp]
        lib.attn_fwd_states.restype = i
        lib.attn_merge_states.argtypes = [vp, vp, vp, i, ctypes.c_longlong, i, vp, vp, vp]
        lib.attn_merge_states.restype = i
        lib.attn_splitkv_workspace_bytes.argtypes = [i, i, i, i, i]
        lib.attn_splitkv_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_splitkv_splits.argtypes = [i, i, i, i]
        lib.attn_splitkv_splits.restype = i
        lib.attn_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, vp, ctypes.c_size_t, vp]
        lib.attn_fwd_splitkv.restype = i
        cache = ctypes.POINTER(AttnCache)
        lib.attn_cache_write.argtypes = [cache, vp, vp, i64p, i64p, vp, i, vp, vp, i, i, vp]
        lib.attn_cache_write.restype = i
        lib.attn_cache_read.argtypes = [cache, vp, vp, vp, i, vp, vp, i, i, vp]
        lib.attn_cache_read.restype = i
        lib.attn_cache_check.argtypes = [vp]
        lib.attn_cache_check.restype = i
        lib.attn_fwd_tree.argtypes = [vp, cache, vp, vp, vp, i, vp, vp, vp, i, i, i, i, f, vp, ctypes.c_size_t, vp]
        lib.attn_fwd_tree.restype = i
        lib.attn_tree_workspace_bytes.argtypes = [i, i, i, i]
        lib.attn_tree_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_qk_rotate.argtypes = [vp, vp, vp, vp, i64p, i64p, i64p, i64p, vp, vp, vp, vp, i, i, vp, vp, i, f, i, i,
                                       i, i, i, vp]
        lib.attn_qk_rotate.restype = i
        lib.attn_fwd_prompt.argtypes = [vp, vp, vp, vp, vp, i64p, i64p, i64p, i64p, vp, vp, i, i, i, i, i, i, i, f, i, vp,
                                        ctypes.c_size_t, vp]
        lib.attn_fwd_prompt.restype = i
        lib.attn_prompt_workspace_bytes.argtypes = [i, i, i, i, i, i]
        lib.attn_prompt_workspace_bytes.restype = ctypes.c_size_t
        lib.attn_cache_weigh.argtypes = [vp, vp, cache, vp, vp, vp, i, vp, vp, i, i, i, f, f, vp]
        lib.attn_cache_weigh.restype = i
        lib.attn_cache_evict.argtypes = [cache, vp, vp, i, vp, i, vp, vp, vp, i, i, i, i, vp]
        lib.attn_cache_evict.restype = i
        _lib = lib
    return _lib


def _check(rc: int):
    if rc != 0:
        raise AttnError(rc, load_library().attn_last_error().decode())


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def attn_fwd_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nk, d, scale, causal, lens_ptr, stream_ptr) -> int:
    """The C call with plain integers for pointers; returns the attn_status code."""
    lib = load_library()
    return lib.attn_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nk, d, scale, int(causal), lens_ptr,
                        stream_ptr)


def _check_qkv(Q, K, V, key_padding_lens):
    """Shapes, dtypes and placement of the inputs; returns (B, H, Nq, Nk, d, lens_ptr)."""
    import torch
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    if K.shape != (B, H, Nk, d) or V.shape != (B, H, Nk, d):
        raise ValueError("K and V must be [B, H, Nk, d] with Q's B, H and d")
    lens_ptr = None
    if key_padding_lens is not None:
        if key_padding_lens.dtype != torch.int32 or not key_padding_lens.is_cuda or key_padding_lens.numel() != B:
            raise ValueError("key_padding_lens must be an int32 CUDA tensor [B]")
        lens_ptr = key_padding_lens.data_ptr()
    return B, H, Nq, Nk, d, lens_ptr


def _outputs(Q, O, LSE):
    import torch
    B, H, Nq, _ = Q.shape
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty((B, H, Nq), dtype=torch.float32, device=Q.device)
    if O.shape != Q.shape or O.dtype != torch.bfloat16 or not O.is_contiguous():
        raise ValueError("O must be a contiguous bf16 tensor shaped like Q")
    if LSE.shape != (B, H, Nq) or LSE.dtype != torch.float32 or not LSE.is_contiguous():
        raise ValueError("LSE must be a contiguous fp32 tensor [B, H, Nq]")
    return O, LSE


def attn_fwd(Q, K, V, O=None, LSE=None, *, scale=None, causal=False, key_padding_lens=None, stream=None,
             rescale_threshold=0.0, exp2_mode=EXP2_DEFAULT, key_block=0):
    """O, LSE = softmax(scale * Q K^T + mask) V and its row logsumexp, on the GPU.

    Q [B,H,Nq,d], K/V [B,H,Nk,d]: contiguous bf16 CUDA tensors.  O (bf16) and LSE
    (fp32 [B,H,Nq]) are allocated when not given.  key_padding_lens: int32 CUDA
    tensor [B] or None.  Enqueued on ``stream`` (default: torch's current stream).
    rescale_threshold / exp2_mode / key_block: the attn_options of attn_fwd_ex (defaults:
    attn_fwd).
    """
    import torch
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    if K.shape != (B, H, Nk, d) or V.shape != (B, H, Nk, d):
        raise ValueError("K and V must be [B, H, Nk, d] with Q's B, H and d")
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty((B, H, Nq), dtype=torch.float32, device=Q.device)
    if O.shape != Q.shape or O.dtype != torch.bfloat16 or not O.is_contiguous():
        raise ValueError("O must be a contiguous bf16 tensor shaped like Q")
    if LSE.shape != (B, H, Nq) or LSE.dtype != torch.float32 or not LSE.is_contiguous():
        raise ValueError("LSE must be a contiguous fp32 tensor [B, H, Nq]")
    lens_ptr = None
    if key_padding_lens is not None:
        if key_padding_lens.dtype != torch.int32 or not key_padding_lens.is_cuda or key_padding_lens.numel() != B:
            raise ValueError("key_padding_lens must be an int32 CUDA tensor [B]")
        lens_ptr = key_padding_lens.data_ptr()
    if rescale_threshold == 0.0 and exp2_mode == EXP2_DEFAULT and key_block == 0:
        rc = attn_fwd_raw(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), B, H, Nq, Nk, d,
                          float(scale), causal, lens_ptr, _stream_handle(stream))
    else:
        opts = AttnOptions(ctypes.sizeof(AttnOptions), float(rescale_threshold), int(exp2_mode), int(key_block))
        rc = load_library().attn_fwd_ex(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), B, H,
                                        Nq, Nk, d, float(scale), int(causal), lens_ptr, ctypes.byref(opts),
                                        _stream_handle(stream))
    _check(rc)
    return O, LSE


def attn_fwd_host(Q, K, V, O, LSE, *, scale=None, causal=False, key_padding_lens=None, stream=None):
    """Host-buffer variant: Q/K/V/O are CPU bf16 tensors (pinned for speed), LSE CPU fp32,
    key_padding_lens a CPU int32 tensor or None.  Blocks until O and LSE are written."""
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    lens_ptr = None if key_padding_lens is None else key_padding_lens.data_ptr()
    lib = load_library()
    rc = lib.attn_fwd_host(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), B, H, Nq, Nk, d,
                           float(scale), int(causal), lens_ptr, _stream_handle(stream))
    _check(rc)
    return O, LSE


def status_sync(stream=None):
    """Synchronise the stream and raise AttnError if a bounded device wait ran out."""
    _check(load_library().attn_status_sync(_stream_handle(stream)))


def release_workspace():
    """Free the workspaces kept for attn_fwd_host and (by every thread) for attn_fwd_tree and attn_fwd_prompt."""
    with _kept_lock:
        for kept in list(_kept_by_threads):
            kept.by_stream.clear()
    _check(load_library().attn_release_workspace())


def version() -> int:
    return load_library().attn_version()


# --- split-KV: partial states and their merge ---------------------------------

def attn_fwd_states(Q, K, V, num_splits, *, scale=None, causal=False, key_padding_lens=None, stream=None):
    """The running states (o~, m, l) of ``num_splits`` key splits (split s covers keys
    [s*C, (s+1)*C), C = 128 * ceil(ceil(Nk/128) / num_splits)).  Returns fp32 CUDA tensors
    o_states [S,B,H,Nq,d], m_states [S,B,H,Nq], l_states [S,B,H,Nq]."""
    import torch
    B, H, Nq, Nk, d, lens_ptr = _check_qkv(Q, K, V, key_padding_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    S = int(num_splits)
    o_st = torch.empty((S, B, H, Nq, d), dtype=torch.float32, device=Q.device)
    m_st = torch.empty((S, B, H, Nq), dtype=torch.float32, device=Q.device)
    l_st = torch.empty((S, B, H, Nq), dtype=torch.float32, device=Q.device)
    rc = load_library().attn_fwd_states(Q.data_ptr(), K.data_ptr(), V.data_ptr(), o_st.data_ptr(), m_st.data_ptr(),
                                        l_st.data_ptr(), B, H, Nq, Nk, d, float(scale), int(causal), lens_ptr, S,
                                        _stream_handle(stream))
    _check(rc)
    return o_st, m_st, l_st


def merge_states(o_states, m_states, l_states, O=None, LSE=None, *, stream=None):
    """Merge S states per row: o_states fp32 [S, ..., d], m_states / l_states fp32 [S, ...].
    Returns O bf16 [..., d] and LSE fp32 [...] (allocated when not given)."""
    import torch
    S, d = o_states.shape[0], o_states.shape[-1]
    rows_shape = tuple(o_states.shape[1:-1])
    for name, t in (("o_states", o_states), ("m_states", m_states), ("l_states", l_states)):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")
    if tuple(m_states.shape) != (S,) + rows_shape or tuple(l_states.shape) != (S,) + rows_shape:
        raise ValueError("m_states and l_states must be [S, ...] matching o_states [S, ..., d]")
    if O is None:
        O = torch.empty(rows_shape + (d,), dtype=torch.bfloat16, device=o_states.device)
    if LSE is None:
        LSE = torch.empty(rows_shape, dtype=torch.float32, device=o_states.device)
    rows = int(math.prod(rows_shape))
    if O.numel() != rows * d or O.dtype != torch.bfloat16 or LSE.numel() != rows or LSE.dtype != torch.float32:
        raise ValueError("O must be bf16 [..., d] and LSE fp32 [...] over the states' rows")
    rc = load_library().attn_merge_states(o_states.data_ptr(), m_states.data_ptr(), l_states.data_ptr(), S, rows, d,
                                          O.data_ptr(), LSE.data_ptr(), _stream_handle(stream))
    _check(rc)
    return O, LSE


def splitkv_splits(B, H, Nq, Nk) -> int:
    """The split count attn_fwd_splitkv picks for num_splits <= 0 on the current device."""
    return load_library().attn_splitkv_splits(B, H, Nq, Nk)


def splitkv_workspace_bytes(B, H, Nq, d, num_splits) -> int:
    return load_library().attn_splitkv_workspace_bytes(B, H, Nq, d, num_splits)


def attn_fwd_splitkv(Q, K, V, O=None, LSE=None, *, num_splits=0, workspace=None, scale=None, causal=False,
                     key_padding_lens=None, stream=None):
    """attn_fwd through split-KV states and their merge.  workspace: a CUDA uint8 tensor
    of at least splitkv_workspace_bytes(...) bytes, allocated here when not given."""
    import torch
    B, H, Nq, Nk, d, lens_ptr = _check_qkv(Q, K, V, key_padding_lens)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    O, LSE = _outputs(Q, O, LSE)
    S = int(num_splits) if num_splits and num_splits > 0 else splitkv_splits(B, H, Nq, Nk)
    need = splitkv_workspace_bytes(B, H, Nq, d, S) if S > 1 else 0
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().attn_fwd_splitkv(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), B, H,
                                         Nq, Nk, d, float(scale), int(causal), lens_ptr, S, ws_ptr, ws_bytes,
                                         _stream_handle(stream))
    _check(rc)
    return O, LSE


# --- other layouts -------------------------------------------------------------

def attn_fwd_strided(Q, K, V, O=None, LSE=None, *, scale=None, causal=False, key_padding_lens=None, stream=None):
    """attn_fwd on 4-D bf16 CUDA tensors viewed as [B, H, N, d] with any strides whose last
    dimension is contiguous (e.g. ``x.transpose(1, 2)`` of a [B, N, H, d] tensor).  O (same
    strides as a new tensor shaped like Q's view when not given) and LSE [B, H, Nq]."""
    import torch
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(3) != 1:
            raise ValueError(f"{name} must be a bf16 CUDA tensor with a contiguous last dimension")
    if K.shape != (B, H, Nk, d) or V.shape != (B, H, Nk, d):
        raise ValueError("K and V must be [B, H, Nk, d] with Q's B, H and d")
    if O is None:
        O = torch.empty((B, Nq, H, d), dtype=torch.bfloat16, device=Q.device).transpose(1, 2)
    if LSE is None:
        LSE = torch.empty((B, H, Nq), dtype=torch.float32, device=Q.device)
    if O.shape != Q.shape or O.dtype != torch.bfloat16 or O.stride(3) != 1:
        raise ValueError("O must be bf16 shaped like Q with a contiguous last dimension")
    lens_ptr = None
    if key_padding_lens is not None:
        lens_ptr = key_padding_lens.data_ptr()

    def st(t):
        return (ctypes.c_int64 * 3)(t.stride(0), t.stride(1), t.stride(2))
    rc = load_library().attn_fwd_strided(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), B, H,
                                         Nq, Nk, d, float(scale), int(causal), lens_ptr, st(Q), st(K), st(V), st(O),
                                         _stream_handle(stream))
    _check(rc)
    return O, LSE


def attn_fwd_varlen(Q, K, V, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, O=None, LSE=None, *, scale=None, causal=False,
                    stream=None):
    """Packed sequences: Q [total_q, H, d], K/V [total_k, H, d] contiguous bf16 CUDA tensors,
    cu_seqlens_q / cu_seqlens_k int32 CUDA tensors [B + 1].  Returns O [total_q, H, d] and
    LSE [H, total_q].  K and V have Q's heads: where a group of query heads shares one, repeat it
    (``K.repeat_interleave(Hq // Hkv, 1)``)."""
    import torch
    total_q, H, d = Q.shape
    total_k = K.shape[0]
    # the library takes one head count, Q's: fewer K/V heads would be read past their end
    if K.shape != (total_k, H, d) or V.shape != (total_k, H, d):
        raise ValueError("K and V must be [total_k, H, d] with Q's H and d (repeat K/V heads that query heads share)")
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.device != Q.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor on Q's device")
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != B + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty((H, total_q), dtype=torch.float32, device=Q.device)
    if O.shape != Q.shape or O.dtype != torch.bfloat16 or O.device != Q.device or not O.is_contiguous():
        raise ValueError("O must be a contiguous bf16 tensor shaped like Q")
    if LSE.shape != (H, total_q) or LSE.dtype != torch.float32 or LSE.device != Q.device or not LSE.is_contiguous():
        raise ValueError("LSE must be a contiguous fp32 tensor [H, total_q]")
    rc = load_library().attn_fwd_varlen(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(),
                                        cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, H, int(max_seqlen_q),
                                        total_q, total_k, d, float(scale), int(causal), _stream_handle(stream))
    _check(rc)
    return O, LSE


# --- paged cache, and attention over it ------------------------------------------
# A decoding step calls these once a layer with little work on the GPU, so the host's time
# counts: the checks are written out in a line each and nothing is looked up twice.

def _cache_args(k_cache, v_cache, k_scale, v_scale):
    """The attn_cache of these tensors (every check of their shapes, types and placement)."""
    import torch
    shape, dtype, dev = k_cache.shape, k_cache.dtype, k_cache.device
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != dtype:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d] of one type")
    if not (k_cache.is_cuda and v_cache.device == dev and k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous CUDA tensors on one device")
    P, H, page, d = shape
    if dtype == torch.bfloat16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache takes no k_scale / v_scale")
        return AttnCache(_CACHE_SIZE, k_cache.data_ptr(), v_cache.data_ptr(), None, None, CACHE_BF16, P, page, H, d)
    if dtype != torch.float8_e4m3fn:
        raise ValueError("the cache must be bf16 or float8_e4m3fn")
    if (k_scale is None or v_scale is None or k_scale.dtype != torch.uint8 or v_scale.dtype != torch.uint8
            or k_scale.shape != shape[:3] or v_scale.shape != shape[:3] or k_scale.device != dev
            or v_scale.device != dev or not k_scale.is_contiguous() or not v_scale.is_contiguous()):
        raise ValueError("k_scale and v_scale must be contiguous uint8 tensors [num_pages, Hkv, page_size] on the "
                         "cache's device")
    return AttnCache(_CACHE_SIZE, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                     CACHE_E4M3, P, page, H, d)


_CACHE_SIZE = ctypes.sizeof(AttnCache)


def _batch_args(dev, block_table, cu_seqlens, lens):
    """Checks the int32 arrays of a batch; returns (B, max_pages, lens pointer)."""
    import torch
    i32 = torch.int32
    if block_table.dim() != 2 or block_table.dtype != i32 or block_table.device != dev or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 tensor [B, max_pages] on the cache's device")
    B, max_pages = block_table.shape
    if cu_seqlens.numel() != B + 1 or cu_seqlens.dtype != i32 or cu_seqlens.device != dev or not cu_seqlens.is_contiguous():
        raise ValueError("the cu_seqlens array must be a contiguous int32 tensor [B + 1] on the cache's device")
    if lens is None:
        return B, max_pages, None
    if lens.numel() != B or lens.dtype != i32 or lens.device != dev or not lens.is_contiguous():
        raise ValueError("start_lens / ctx_lens must be a contiguous int32 tensor [B] on the cache's device")
    return B, max_pages, lens.data_ptr()


def _elsewhere(dev, stream):
    """Context that makes a call's device current, and its stream for what is allocated there
    (so that buffers made here belong to the stream that uses them); None when both already are."""
    import torch
    if dev.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    if stream is None:
        return None if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError("stream is on another device than the tensors")
    import contextlib
    both = contextlib.ExitStack()
    both.enter_context(torch.cuda.device(dev))
    both.enter_context(torch.cuda.stream(stream))
    return both


def attn_cache_write(K, V, k_cache, v_cache, block_table, cu_seqlens, *, start_lens=None, k_scale=None, v_scale=None,
                     stream=None):
    """Put packed new tokens into a paged cache, in place.

    K, V [total, Hkv, d]: bf16 CUDA tensors with a contiguous last dimension (views of a joint
    projection need no copy).  k_cache, v_cache [num_pages, Hkv, page_size, d] (page_size a
    multiple of 16 up to 65536): bf16 or float8_e4m3fn; an e4m3 cache comes with k_scale and
    v_scale, uint8 [num_pages, Hkv, page_size] (value = code * 2^(s - 127)).  block_table int32
    [B, max_pages]; cu_seqlens int32 [B + 1]: sequence b's tokens are rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1 and go to positions start_lens[b], ... (int32 [B]; None: 0).  Tokens
    without a page are left out and reported by cache_check().
    """
    import torch
    dev = k_cache.device
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return attn_cache_write(K, V, k_cache, v_cache, block_table, cu_seqlens, start_lens=start_lens,
                                    k_scale=k_scale, v_scale=v_scale)
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    shape = K.shape
    if (len(shape) != 3 or shape[1] != cache.num_heads or shape[2] != cache.d or V.shape != shape
            or K.dtype != torch.bfloat16 or V.dtype != torch.bfloat16 or K.device != dev or V.device != dev):
        raise ValueError("K and V must be bf16 tensors [total, Hkv, d] on the cache's device")
    ks, vs = K.stride(), V.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("K and V must have a contiguous last dimension")
    B, max_pages, start_ptr = _batch_args(dev, block_table, cu_seqlens, start_lens)
    kst = _Strides(ks[0], ks[1])
    rc = load_library().attn_cache_write(cache, K.data_ptr(), V.data_ptr(), kst,
                                         kst if vs == ks else _Strides(vs[0], vs[1]), block_table.data_ptr(),
                                         max_pages, cu_seqlens.data_ptr(), start_ptr, B, shape[0],
                                         torch._C._cuda_getCurrentRawStream(dev.index))
    if rc != 0:
        _check(rc)


_Strides = ctypes.c_int64 * 2


def attn_cache_read(k_cache, v_cache, block_table, cu_seqlens, total, K=None, V=None, *, start_lens=None, k_scale=None,
                    v_scale=None, stream=None):
    """Cached positions as packed bf16 K, V [total, Hkv, d] (allocated when not given), the
    layout attn_fwd_varlen takes where every query head has its own K/V head; for grouped heads
    repeat them (``K.repeat_interleave(Hq // Hkv, 1)``).  Row cu_seqlens[b] + i is position
    start_lens[b] + i of sequence b; rows outside every sequence are left as they were, positions without a page are
    zeros and reported by cache_check().  The cache's arguments: as attn_cache_write."""
    import torch
    dev = k_cache.device
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return attn_cache_read(k_cache, v_cache, block_table, cu_seqlens, total, K, V, start_lens=start_lens,
                                   k_scale=k_scale, v_scale=v_scale)
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    B, max_pages, start_ptr = _batch_args(dev, block_table, cu_seqlens, start_lens)
    total = int(total)
    shape = (total, cache.num_heads, cache.d)
    if K is None:
        K = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if V is None:
        V = torch.empty_like(K)
    for t in (K, V):
        if t.shape != shape or t.dtype != torch.bfloat16 or t.device != dev or not t.is_contiguous():
            raise ValueError("K and V must be contiguous bf16 tensors [total, Hkv, d] on the cache's device")
    rc = load_library().attn_cache_read(cache, K.data_ptr(), V.data_ptr(), block_table.data_ptr(), max_pages,
                                        cu_seqlens.data_ptr(), start_ptr, B, total,
                                        torch._C._cuda_getCurrentRawStream(dev.index))
    if rc != 0:
        _check(rc)
    return K, V


def tree_workspace_bytes(Hq, Hkv, max_seqlen_q, d) -> int:
    """Bytes of workspace attn_fwd_tree needs (0 for invalid arguments)."""
    return load_library().attn_tree_workspace_bytes(Hq, Hkv, max_seqlen_q, d)


class _Kept:
    """A host thread's workspaces: (device index, stream) -> uint8 tensor.  They go with the thread."""
    __slots__ = ("by_stream", "__weakref__")

    def __init__(self):
        self.by_stream = {}


_thread = threading.local()
_kept_by_threads = weakref.WeakSet()  # for release_workspace
_kept_lock = threading.Lock()


def _tree_workspace(nbytes, dev, raw):
    """attn_fwd_tree's and attn_fwd_prompt's default workspace: one kept for each stream and host thread, whose calls run
    one after the other (two threads may interleave their launches on a stream), until the thread
    ends; a captured call gets its own, which belongs to the graph (graphs may run at once)."""
    import torch
    if torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    kept = getattr(_thread, "kept", None)
    if kept is None:
        kept = _thread.kept = _Kept()
        with _kept_lock:
            _kept_by_threads.add(kept)
    ws = kept.by_stream.get((dev.index, raw))
    if ws is None or ws.numel() < nbytes:
        ws = kept.by_stream[dev.index, raw] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws


def attn_fwd_tree(Q, k_cache, v_cache, block_table, ctx_lens, cu_seqlens_q, max_seqlen_q, O=None, LSE=None, *,
                  tree_mask=None, k_scale=None, v_scale=None, scale=None, workspace=None, stream=None):
    """Attention of each sequence's new (drafted) tokens over its paged cache.

    Q [total_q, Hq, d]: contiguous bf16 CUDA tensor, sequence b's tokens at rows
    cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1 (int32 [B + 1]), at most max_seqlen_q <= 64 of
    them; their K and V are already cached at positions ctx_lens[b], ... (int32 [B]; None: 0).
    Hq is a multiple of the cache's heads, at most 65536; O may be Q.  tree_mask int64 [total_q]:
    bit u of a token's word lets it see token u of its sequence (None: a chain, u <= i); every
    token sees the context.  One token per sequence is plain decoding.  Returns O
    [total_q, Hq, d] and LSE [Hq, total_q] (allocated when not given).  workspace: a CUDA uint8
    tensor of tree_workspace_bytes(...) that no other call in flight uses; when not given, one
    kept for the stream and host thread until the thread ends (a captured call gets its own;
    release_workspace() lets them go).  The cache's arguments: as attn_cache_write.
    """
    import torch
    dev = k_cache.device
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return attn_fwd_tree(Q, k_cache, v_cache, block_table, ctx_lens, cu_seqlens_q, max_seqlen_q, O, LSE,
                                 tree_mask=tree_mask, k_scale=k_scale, v_scale=v_scale, scale=scale,
                                 workspace=workspace)
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    shape = Q.shape
    if (len(shape) != 3 or shape[2] != cache.d or Q.dtype != torch.bfloat16 or Q.device != dev
            or not Q.is_contiguous()):
        raise ValueError("Q must be a contiguous bf16 tensor [total_q, Hq, d] on the cache's device")
    total_q, Hq, d = shape
    max_seqlen_q = int(max_seqlen_q)
    B, max_pages, ctx_ptr = _batch_args(dev, block_table, cu_seqlens_q, ctx_lens)
    mask_ptr = None
    if tree_mask is not None:
        if (tree_mask.dtype != torch.int64 or tree_mask.device != dev or tree_mask.numel() != total_q
                or not tree_mask.is_contiguous()):
            raise ValueError("tree_mask must be a contiguous int64 tensor [total_q] on the cache's device")
        mask_ptr = tree_mask.data_ptr()
    lib = load_library()
    if O is None:
        O = torch.empty_like(Q)
    elif O.shape != shape or O.dtype != torch.bfloat16 or O.device != dev or not O.is_contiguous():
        raise ValueError("O must be a contiguous bf16 tensor shaped like Q")
    if LSE is None:
        LSE = torch.empty((Hq, total_q), dtype=torch.float32, device=dev)
    elif LSE.shape != (Hq, total_q) or LSE.dtype != torch.float32 or LSE.device != dev or not LSE.is_contiguous():
        raise ValueError("LSE must be a contiguous fp32 tensor [Hq, total_q]")
    raw = torch._C._cuda_getCurrentRawStream(dev.index)
    if workspace is None:
        nbytes = lib.attn_tree_workspace_bytes(Hq, cache.num_heads, max_seqlen_q, d)
        workspace = _tree_workspace(nbytes, dev, raw)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    else:
        nbytes = workspace.numel() * workspace.element_size()
    rc = lib.attn_fwd_tree(Q.data_ptr(), cache, O.data_ptr(), LSE.data_ptr(), block_table.data_ptr(), max_pages,
                           cu_seqlens_q.data_ptr(), ctx_ptr, mask_ptr, B, Hq, max_seqlen_q, total_q,
                           1.0 / math.sqrt(d) if scale is None else scale, workspace.data_ptr(), nbytes, raw)
    if rc != 0:
        _check(rc)
    return O, LSE


# --- prompts of grouped heads, and a cache of bounded length -----------------------

WEIGHT_BF16, WEIGHT_FP32 = 0, 1


@functools.lru_cache(maxsize=256)
def _strides(row, head):
    """A pair of strides as the library takes them (never written to)."""
    return _Strides(row, head)


def _packed(name, t, dev, heads=None, d=None):
    """Checks a packed bf16 tensor [total, heads, d] with a contiguous last dimension; returns its strides."""
    import torch
    shape = t.shape
    if (len(shape) != 3 or t.dtype != torch.bfloat16 or t.device != dev or (heads is not None and shape[1] != heads)
            or (d is not None and shape[2] != d)):
        raise ValueError(f"{name} must be a bf16 tensor [total, heads, d] with the call's heads and d, on its device")
    st = t.stride()
    if st[2] != 1 and t.numel():
        raise ValueError(f"{name} must have a contiguous last dimension")
    return _strides(st[0], st[1])


def attn_qk_rotate(Q, K, cu_seqlens=None, inv_freq=None, Q_out=None, K_out=None, *, start_lens=None, positions=None,
                   q_weight=None, k_weight=None, eps=1e-6, interleaved=False, stream=None):
    """Norms of query and key heads and their rotation by position, in one pass.

    Q [total, Hq, d], K [total, Hkv, d]: bf16 CUDA tensors with a contiguous last dimension (views of a
    joint projection need no copy).  q_weight, k_weight [d] (bf16 or fp32, both alike; None: no norm):
    x * w / sqrt(mean(x^2) + eps).  inv_freq fp32 [r], r a multiple of 8 up to d / 2 (None: no
    rotation): column i turns with column i + r (interleaved: 2 i with 2 i + 1) by position *
    inv_freq[i].  cu_seqlens int32 [B + 1] (None: all rows are one sequence): row cu_seqlens[b] + i is at
    start_lens[b] + i (int32 [B]; None: 0), rows outside every sequence are left as they were;
    positions int32 [total] replaces these.  Returns Q_out and K_out (allocated contiguous when not
    given; Q_out may be Q and K_out K, an output overlaps no other input).
    """
    import torch
    dev = Q.device
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return attn_qk_rotate(Q, K, cu_seqlens, inv_freq, Q_out, K_out, start_lens=start_lens, positions=positions,
                                  q_weight=q_weight, k_weight=k_weight, eps=eps, interleaved=interleaved)
    qs = _packed("Q", Q, dev)
    total, Hq, d = Q.shape
    ks = _packed("K", K, dev, None, d)
    Hkv = K.shape[1]
    if K.shape[0] != total:
        raise ValueError("Q and K must have the same tokens")
    i32 = torch.int32
    B, cu_ptr, start_ptr, pos_ptr, freq_ptr, r = 1, None, None, None, None, 0
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        if B < 0 or cu_seqlens.dtype != i32 or cu_seqlens.device != dev or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous int32 tensor [B + 1] on Q's device")
        cu_ptr = cu_seqlens.data_ptr()
    if start_lens is not None:
        if start_lens.numel() != B or start_lens.dtype != i32 or start_lens.device != dev or not start_lens.is_contiguous():
            raise ValueError("start_lens must be a contiguous int32 tensor [B] on Q's device")
        start_ptr = start_lens.data_ptr()
    if positions is not None:
        if positions.numel() != total or positions.dtype != i32 or positions.device != dev or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous int32 tensor [total] on Q's device")
        pos_ptr = positions.data_ptr()
    if inv_freq is not None:
        if inv_freq.dim() != 1 or inv_freq.dtype != torch.float32 or inv_freq.device != dev or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous fp32 tensor [r] on Q's device")
        freq_ptr, r = inv_freq.data_ptr(), inv_freq.numel()
    wtype, wptr = WEIGHT_BF16, [None, None]
    for i, w in enumerate((q_weight, k_weight)):
        if w is None:
            continue
        if (w.numel() != d or w.dtype not in (torch.bfloat16, torch.float32) or w.device != dev or not w.is_contiguous()
                or (i == 1 and q_weight is not None and w.dtype != q_weight.dtype)):
            raise ValueError("q_weight and k_weight must be contiguous tensors [d] of one type, bf16 or fp32, on Q's device")
        wtype = WEIGHT_FP32 if w.dtype == torch.float32 else WEIGHT_BF16
        wptr[i] = w.data_ptr()
    if Q_out is None:
        Q_out, qos = torch.empty((total, Hq, d), dtype=torch.bfloat16, device=dev), _strides(Hq * d, d)
    else:
        qos = _packed("Q_out", Q_out, dev, Hq, d)
    if K_out is None:
        K_out, kos = torch.empty((total, Hkv, d), dtype=torch.bfloat16, device=dev), _strides(Hkv * d, d)
    else:
        kos = _packed("K_out", K_out, dev, Hkv, d)
    if Q_out.shape[0] != total or K_out.shape[0] != total:
        raise ValueError("Q_out and K_out must be shaped like Q and K")
    rc = load_library().attn_qk_rotate(Q.data_ptr(), K.data_ptr(), Q_out.data_ptr(), K_out.data_ptr(), qs, ks, qos, kos,
                                       cu_ptr, start_ptr, pos_ptr, freq_ptr, r, 1 if interleaved else 0, wptr[0], wptr[1],
                                       wtype, eps, B, Hq, Hkv, d, total, torch._C._cuda_getCurrentRawStream(dev.index))
    if rc != 0:
        _check(rc)
    return Q_out, K_out


def prompt_workspace_bytes(B, Hq, max_seqlen_q, total_q, total_k, d) -> int:
    """Bytes of workspace with which attn_fwd_prompt splits keys (0: it does not, or invalid arguments)."""
    return load_library().attn_prompt_workspace_bytes(B, Hq, max_seqlen_q, total_q, total_k, d)


def attn_fwd_prompt(Q, K, V, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, O=None, LSE=None, *, workspace=None, scale=None,
                    causal=True, stream=None):
    """Attention of packed prompts whose query heads share K/V heads.

    Q [total_q, Hq, d], K, V [total_k, Hkv, d]: bf16 CUDA tensors with a contiguous last dimension
    (views of a joint projection need no copy), Hq a multiple of Hkv; cu_seqlens_q / cu_seqlens_k int32
    [B + 1]; max_seqlen_q >= the longest sequence's queries.  causal: bottom-right aligned, so more keys
    than queries are a prompt over its prefix.  Returns O [total_q, Hq, d] and LSE [Hq, total_q]
    (allocated when not given; rows outside every sequence are left as they were).  What K and V hold
    where a row does not look does not reach it.  Few tiles of 128 queries over many keys are split along
    the keys, in a workspace: a uint8 tensor of prompt_workspace_bytes(...) that no other call in flight
    uses; when not given, the stream's own is used, as in attn_fwd_tree.
    """
    import torch
    dev = Q.device
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return attn_fwd_prompt(Q, K, V, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, O, LSE, workspace=workspace,
                                   scale=scale, causal=causal)
    qs = _packed("Q", Q, dev)
    total_q, Hq, d = Q.shape
    ks = _packed("K", K, dev, None, d)
    total_k, Hkv = K.shape[:2]
    vs = _packed("V", V, dev, Hkv, d)
    if V.shape[0] != total_k:
        raise ValueError("K and V must have the same tokens")
    B = cu_seqlens_q.numel() - 1
    for t in (cu_seqlens_q, cu_seqlens_k):
        if B < 0 or t.numel() != B + 1 or t.dtype != torch.int32 or t.device != dev or not t.is_contiguous():
            raise ValueError("cu_seqlens_q and cu_seqlens_k must be contiguous int32 tensors [B + 1] on Q's device")
    if O is None:
        O, os_ = torch.empty((total_q, Hq, d), dtype=torch.bfloat16, device=dev), _strides(Hq * d, d)
    else:
        os_ = _packed("O", O, dev, Hq, d)
        if O.shape[0] != total_q:
            raise ValueError("O must be shaped like Q")
    if LSE is None:
        LSE = torch.empty((Hq, total_q), dtype=torch.float32, device=dev)
    elif LSE.shape != (Hq, total_q) or LSE.dtype != torch.float32 or LSE.device != dev or not LSE.is_contiguous():
        raise ValueError("LSE must be a contiguous fp32 tensor [Hq, total_q]")
    lib, raw, max_q = load_library(), torch._C._cuda_getCurrentRawStream(dev.index), int(max_seqlen_q)
    if workspace is None:
        nbytes = lib.attn_prompt_workspace_bytes(B, Hq, max_q, total_q, total_k, d)
        if nbytes:
            workspace = _tree_workspace(nbytes, dev, raw)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on Q's device")
    rc = lib.attn_fwd_prompt(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), qs, ks, vs, os_,
                             cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Hq, Hkv, max_q, total_q, total_k, d,
                             1.0 / math.sqrt(d) if scale is None else scale, 1 if causal else 0,
                             None if workspace is None else workspace.data_ptr(),
                             0 if workspace is None else workspace.numel(), raw)
    if rc != 0:
        _check(rc)
    return O, LSE


def _pool_weights(name, w, shape, dev):
    import torch
    if w.dtype != torch.float32 or w.shape != shape or w.device != dev or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor [num_pages, Hkv, page_size] on the cache's device")


def attn_cache_weigh(Q, LSE, k_cache, weights, block_table, ctx_lens, cu_seqlens_q, out=None, *, decay=1.0, k_scale=None,
                     scale=None, stream=None):
    """The attention weight that cached keys receive from these queries, added to what they had.

    Q [total_q, Hq, d] and LSE [Hq, total_q]: queries and what their attention returned (attn_fwd_tree,
    attn_fwd_prompt, attn_fwd_varlen; same scale); cu_seqlens_q int32 [B + 1], any number of tokens a
    sequence, whose keys are cached at positions ctx_lens[b], ... (int32 [B]; None: 0); token i sees
    positions up to ctx_lens[b] + i.  weights, out fp32 [num_pages, Hkv, page_size]:
    out = decay * weights + sum over the rows that see a key of exp(scale * q . k - LSE), where positions
    that the call brought start from 0; decay = 0 reads no weights (they may be None).  Only positions of
    sequences with tokens are written.  Returns out (None: weights, in place).  The cache's other
    arguments: as attn_cache_write; its values are not needed.
    """
    import torch
    dev = k_cache.device
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return attn_cache_weigh(Q, LSE, k_cache, weights, block_table, ctx_lens, cu_seqlens_q, out, decay=decay,
                                    k_scale=k_scale, scale=scale)
    cache = _cache_args(k_cache, k_cache, k_scale, k_scale)
    shape = Q.shape
    if (len(shape) != 3 or shape[2] != cache.d or Q.dtype != torch.bfloat16 or Q.device != dev or not Q.is_contiguous()):
        raise ValueError("Q must be a contiguous bf16 tensor [total_q, Hq, d] on the cache's device")
    total_q, Hq, d = shape
    if LSE.shape != (Hq, total_q) or LSE.dtype != torch.float32 or LSE.device != dev or not LSE.is_contiguous():
        raise ValueError("LSE must be a contiguous fp32 tensor [Hq, total_q] on the cache's device")
    B, max_pages, ctx_ptr = _batch_args(dev, block_table, cu_seqlens_q, ctx_lens)
    if out is None:
        out = weights
    if out is None or (weights is None and decay != 0):
        raise ValueError("weights may be None only with decay = 0 and an out")
    pool = k_cache.shape[:3]
    _pool_weights("out", out, pool, dev)
    if weights is not None and weights is not out:
        _pool_weights("weights", weights, pool, dev)
    rc = load_library().attn_cache_weigh(Q.data_ptr(), LSE.data_ptr(), cache, None if weights is None else weights.data_ptr(),
                                         out.data_ptr(), block_table.data_ptr(), max_pages, cu_seqlens_q.data_ptr(), ctx_ptr,
                                         B, Hq, total_q, 1.0 / math.sqrt(d) if scale is None else scale, decay,
                                         torch._C._cuda_getCurrentRawStream(dev.index))
    if rc != 0:
        _check(rc)
    return out


def attn_cache_evict(k_cache, v_cache, weights, block_table, lens, keep, *, sink=0, recent=0, out_table=None, kept=None,
                     out_lens=None, k_scale=None, v_scale=None, stream=None):
    """Cut sequences to ``keep`` tokens a head by their weights; their rows are packed in order.

    lens int32 [B]: the sequences' tokens; weights fp32 [num_pages, Hkv, page_size] (attn_cache_weigh).  A
    longer sequence keeps, in each head, its first ``sink`` tokens, its last ``recent`` ones and the
    largest weights between (the first of equal ones).  K, V, scales and weights of what is kept move to
    positions 0, 1, ... of the pages of out_table (int32 [B, out_max_pages], pages that no sequence of the
    call reads) or, without one, of the sequence's own.  Returns kept int32 [B, Hkv, keep] (the positions,
    increasing; -1 past the sequence's tokens) and out_lens int32 [B] = min(lens, keep; no part of lens),
    allocated when not given.  Positions without a page are reported by cache_check().  The cache's arguments: as
    attn_cache_write.
    """
    import torch
    dev = k_cache.device
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return attn_cache_evict(k_cache, v_cache, weights, block_table, lens, keep, sink=sink, recent=recent,
                                    out_table=out_table, kept=kept, out_lens=out_lens, k_scale=k_scale, v_scale=v_scale)
    cache = _cache_args(k_cache, v_cache, k_scale, v_scale)
    _pool_weights("weights", weights, k_cache.shape[:3], dev)
    i32 = torch.int32
    if block_table.dim() != 2 or block_table.dtype != i32 or block_table.device != dev or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 tensor [B, max_pages] on the cache's device")
    B, max_pages = block_table.shape
    if lens.numel() != B or lens.dtype != i32 or lens.device != dev or not lens.is_contiguous():
        raise ValueError("lens must be a contiguous int32 tensor [B] on the cache's device")
    to_ptr, to_pages = None, 0
    if out_table is not None:
        if (out_table.dim() != 2 or out_table.shape[0] != B or out_table.dtype != i32 or out_table.device != dev
                or not out_table.is_contiguous()):
            raise ValueError("out_table must be a contiguous int32 tensor [B, out_max_pages] on the cache's device")
        to_ptr, to_pages = out_table.data_ptr(), out_table.shape[1]
    keep = int(keep)
    if kept is None:
        kept = torch.empty((B, cache.num_heads, max(keep, 0)), dtype=i32, device=dev)
    elif kept.shape != (B, cache.num_heads, keep) or kept.dtype != i32 or kept.device != dev or not kept.is_contiguous():
        raise ValueError("kept must be a contiguous int32 tensor [B, Hkv, keep] on the cache's device")
    if out_lens is None:
        out_lens = torch.empty(B, dtype=i32, device=dev)
    elif out_lens.numel() != B or out_lens.dtype != i32 or out_lens.device != dev or not out_lens.is_contiguous():
        raise ValueError("out_lens must be a contiguous int32 tensor [B] on the cache's device")
    rc = load_library().attn_cache_evict(cache, weights.data_ptr(), block_table.data_ptr(), max_pages, to_ptr, to_pages,
                                         lens.data_ptr(), kept.data_ptr(), out_lens.data_ptr(), B, keep, int(sink),
                                         int(recent), torch._C._cuda_getCurrentRawStream(dev.index))
    if rc != 0:
        _check(rc)
    return kept, out_lens


def cache_check(stream=None):
    """Synchronise the stream; AttnError if a wait ran out or a cache call met a position without a page."""
    _check(load_library().attn_cache_check(_stream_handle(stream)))


# --- the CPU library (libattn_cpu.so, include/attn_cpu.h) ------------------------

CPU_LIB_PATH = os.path.join(_HERE, "libattn_cpu.so")
CPU_EXPORTS = ("attn_fwd_cpu",)
_cpu_lib = None


def load_cpu_library():
    """Load libattn_cpu.so (built by __graft_entry__.build()); raises if it is absent."""
    global _cpu_lib
    if _cpu_lib is None:
        if not os.path.exists(CPU_LIB_PATH):
            raise ImportError(f"{CPU_LIB_PATH} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(CPU_LIB_PATH)
        vp, i = ctypes.c_void_p, ctypes.c_int
        lib.attn_fwd_cpu.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, ctypes.c_float, i, vp, i]
        lib.attn_fwd_cpu.restype = i
        _cpu_lib = lib
    return _cpu_lib


def attn_fwd_cpu(Q, K, V, *, scale=None, causal=False, key_padding_lens=None, num_threads=0):
    """The forward on the host CPU.  Q [B,H,Nq,d], K/V [B,H,Nk,d]: numpy uint16 arrays of
    bf16 codes.  Returns O (uint16 codes, same shape as Q) and LSE (float32 [B,H,Nq])."""
    import numpy as np
    Q, K, V = (np.ascontiguousarray(a, dtype=np.uint16) for a in (Q, K, V))
    B, H, Nq, d = Q.shape
    Nk = K.shape[2]
    if K.shape != (B, H, Nk, d) or V.shape != (B, H, Nk, d):
        raise ValueError("K and V must be [B, H, Nk, d] with Q's B, H and d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    O = np.empty_like(Q)
    LSE = np.empty((B, H, Nq), dtype=np.float32)
    lens = None if key_padding_lens is None else np.ascontiguousarray(key_padding_lens, dtype=np.int32)
    rc = load_cpu_library().attn_fwd_cpu(Q.ctypes.data, K.ctypes.data if Nk else None, V.ctypes.data if Nk else None,
                                         O.ctypes.data, LSE.ctypes.data, B, H, Nq, Nk, d, float(scale), int(causal),
                                         None if lens is None else lens.ctypes.data, int(num_threads))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_cpu failed")
    return O, LSE
