"""Thin Python binding of the C ABI in include/kda.h (argument marshalling only).

Every step of the computation runs in the CUDA kernels of ``_build/libkda.so``
(or, inside ``using_library(load_debug_library())``, of its bounds-checking
debug build); PyTorch only provides device memory and the current stream.
There is no CPU fallback: if the library is missing or no GPU is present,
calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from itertools import accumulate
from typing import NamedTuple, Optional

import torch

from . import build as _build

KDA_OK = 0
STATUS_NAMES = {0: "KDA_OK", -1: "KDA_ERR_INVALID_ARG", -2: "KDA_ERR_UNSUPPORTED", -3: "KDA_ERR_CUDA",
                -4: "KDA_ERR_CKPT_OVERFLOW", -5: "KDA_ERR_WORKSPACE", -6: "KDA_ERR_TIMEOUT",
                -7: "KDA_ERR_BOUNDS"}
STATUS_CODES = {v: k for k, v in STATUS_NAMES.items()}
DTYPE_BF16, DTYPE_FP32, DTYPE_E4M3 = 0, 1, 2   # (e4m3: attention caches only)

# Every symbol include/kda.h declares.
EXPORTS = ("kda_prefill_workspace_size", "kda_prefill_launch_count", "kda_prefill", "kda_prefill_status",
           "kda_prefill_pooled", "kda_prefill_fused", "kda_decode", "kda_decode_fused", "kda_decode_paged",
           "kda_decode_multi", "kda_prefill_noalloc", "kda_gdn_workspace_size", "kda_gdn_prefill",
           "kda_gdn_prefill_pooled", "kda_gdn_decode", "kda_gdn_decode_multi", "kda_plan_batch", "kda_kv_append",
           "kda_attn_workspace_size", "kda_attn_decode_workspace_size", "kda_attn_prefill", "kda_attn_prefill_paged", "kda_attn_decode", "kda_last_error",
           "kda_version")

# Size of the library's built-in scratch array used by kda_prefill_noalloc.
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class KDAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


class PrefillDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("num_heads", ctypes.c_int32), ("head_dim_k", ctypes.c_int32),
                ("head_dim_v", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("ckpt_stride", ctypes.c_int32),
                ("ckpt_capacity", ctypes.c_int64), ("max_seq_len", ctypes.c_int64),
                ("segment_chunks", ctypes.c_int32), ("scalar_gate", ctypes.c_int32),
                ("recurrence_ctas", ctypes.c_int32), ("conv_width", ctypes.c_int32),
                ("conv_silu", ctypes.c_int32), ("wait_limit", ctypes.c_uint32)]


class GdnDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("num_qk_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_dim_k", ctypes.c_int32), ("head_dim_v", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("ckpt_stride", ctypes.c_int32), ("ckpt_capacity", ctypes.c_int64),
                ("max_seq_len", ctypes.c_int64), ("wait_limit", ctypes.c_uint32)]


class AppendDesc(ctypes.Structure):
    _fields_ = [("total_tokens", ctypes.c_int64), ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("rope_scale", ctypes.c_float),
                ("num_seqs", ctypes.c_int32), ("page_size", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int64), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("page_size", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("max_seq_len", ctypes.c_int64), ("scale", ctypes.c_float),
                ("wait_limit", ctypes.c_uint32)]


class BatchPlan(NamedTuple):
    """Device tables of one batch (``plan_batch``), all int32."""
    cu_seqlens: torch.Tensor     # [N + 1] token offsets
    init_slots: torch.Tensor     # [N] slot each request starts from, -1: zeros
    state_slots: torch.Tensor    # [N] slot its state ends in
    ckpt_offsets: torch.Tensor   # [N + 1] its first snapshot
    ckpt_slots: torch.Tensor     # [ckpt_capacity] slot of each snapshot, -1: not taken
    seq_ids: torch.Tensor        # [total_tokens] request of each row, -1: padding
    positions: torch.Tensor      # [total_tokens] its position in the request
    free_head: torch.Tensor      # [1] entries of free_slots used up


_lib = None
_vp = ctypes.c_void_p


def default_library_path() -> str:
    """libkda.so, or its bounds-checking debug build when the environment
    variable KDA_LIBRARY is "debug" (every call of the binding then runs with
    the index checks, and one that fails raises KDAError KDA_ERR_BOUNDS)."""
    if os.environ.get("KDA_LIBRARY", "") == "debug":
        return _build.debug_library_path()
    return _build.library_path()


def load_library(path: Optional[str] = None):
    """Load the library (default_library_path() unless `path` is given; raises
    if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or default_library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with linear_attention_serving_k1_gb300.build.build()")
    lib = ctypes.CDLL(path)
    lib.kda_prefill_workspace_size.restype = ctypes.c_size_t
    lib.kda_prefill_workspace_size.argtypes = [ctypes.POINTER(PrefillDesc)]
    lib.kda_prefill_launch_count.restype = ctypes.c_int32
    lib.kda_prefill_launch_count.argtypes = [ctypes.POINTER(PrefillDesc)]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill.argtypes = [_vp] * 10 + [ctypes.POINTER(PrefillDesc), _vp, ctypes.c_size_t, _vp]
    lib.kda_prefill_status.restype = ctypes.c_int
    lib.kda_prefill_status.argtypes = [_vp, _vp]
    lib.kda_decode.restype = ctypes.c_int
    lib.kda_decode.argtypes = [_vp] * 7 + [ctypes.c_int32] * 5 + [_vp]
    lib.kda_prefill_fused.restype = ctypes.c_int
    lib.kda_prefill_fused.argtypes = [_vp] * 14 + [ctypes.POINTER(PrefillDesc), _vp, ctypes.c_size_t, _vp]
    lib.kda_decode_fused.restype = ctypes.c_int
    lib.kda_decode_fused.argtypes = [_vp] * 10 + [ctypes.c_int32] * 7 + [_vp]
    lib.kda_prefill_pooled.restype = ctypes.c_int
    lib.kda_prefill_pooled.argtypes = [_vp] * 8 + [ctypes.c_int64, _vp, _vp, _vp, ctypes.POINTER(PrefillDesc),
                                                   _vp, ctypes.c_size_t, _vp]
    lib.kda_decode_paged.restype = ctypes.c_int
    lib.kda_decode_paged.argtypes = [_vp] * 6 + [ctypes.c_int64, _vp, _vp] + [ctypes.c_int32] * 5 + [_vp, _vp]
    lib.kda_decode_multi.restype = ctypes.c_int
    lib.kda_decode_multi.argtypes = ([_vp] * 6 + [ctypes.c_int64, _vp, _vp, _vp] + [ctypes.c_int32] * 6 +
                                     [_vp, _vp])
    lib.kda_prefill_noalloc.restype = ctypes.c_int
    lib.kda_prefill_noalloc.argtypes = [_vp] * 10 + [ctypes.POINTER(PrefillDesc), _vp]
    lib.kda_gdn_workspace_size.restype = ctypes.c_size_t
    lib.kda_gdn_workspace_size.argtypes = [ctypes.POINTER(GdnDesc)]
    lib.kda_gdn_prefill.restype = ctypes.c_int
    lib.kda_gdn_prefill.argtypes = [_vp] * 10 + [ctypes.POINTER(GdnDesc), _vp, ctypes.c_size_t, _vp]
    lib.kda_gdn_prefill_pooled.restype = ctypes.c_int
    lib.kda_gdn_prefill_pooled.argtypes = [_vp] * 8 + [ctypes.c_int64, _vp, _vp, _vp, ctypes.POINTER(GdnDesc),
                                                       _vp, ctypes.c_size_t, _vp]
    lib.kda_gdn_decode.restype = ctypes.c_int
    lib.kda_gdn_decode.argtypes = [_vp] * 6 + [ctypes.c_int64, _vp, _vp] + [ctypes.c_int32] * 6 + [_vp, _vp]
    lib.kda_gdn_decode_multi.restype = ctypes.c_int
    lib.kda_gdn_decode_multi.argtypes = ([_vp] * 6 + [ctypes.c_int64, _vp, _vp, _vp] + [ctypes.c_int32] * 7 +
                                         [_vp, _vp])
    lib.kda_plan_batch.restype = ctypes.c_int
    lib.kda_plan_batch.argtypes = ([_vp] * 5 + [ctypes.c_int32, _vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                                ctypes.c_int64, _vp, ctypes.c_int32] + [_vp] * 10)
    lib.kda_kv_append.restype = ctypes.c_int
    lib.kda_kv_append.argtypes = [_vp] * 14 + [ctypes.POINTER(AppendDesc), _vp]
    lib.kda_attn_workspace_size.restype = ctypes.c_size_t
    lib.kda_attn_workspace_size.argtypes = [ctypes.POINTER(AttnDesc)]
    lib.kda_attn_decode_workspace_size.restype = ctypes.c_size_t
    lib.kda_attn_decode_workspace_size.argtypes = [ctypes.POINTER(AttnDesc)]
    lib.kda_attn_prefill.restype = ctypes.c_int
    lib.kda_attn_prefill.argtypes = [_vp] * 6 + [ctypes.POINTER(AttnDesc), _vp, ctypes.c_size_t, _vp]
    lib.kda_attn_prefill_paged.restype = ctypes.c_int
    lib.kda_attn_prefill_paged.argtypes = [_vp] * 10 + [ctypes.POINTER(AttnDesc), _vp, ctypes.c_size_t, _vp]
    lib.kda_attn_decode.restype = ctypes.c_int
    lib.kda_attn_decode.argtypes = [_vp] * 9 + [ctypes.POINTER(AttnDesc), _vp, _vp, ctypes.c_size_t, _vp]
    lib.kda_last_error.restype = ctypes.c_char_p
    lib.kda_last_error.argtypes = []
    lib.kda_version.restype = ctypes.c_int32
    lib.kda_version.argtypes = []
    if path == default_library_path():
        _lib = lib
    return lib


def load_debug_library():
    """Load the debug build libkda_debug.so (same ABI; every data-dependent
    global index checked, failures returned as KDA_ERR_BOUNDS)."""
    return load_library(_build.debug_library_path())


@contextlib.contextmanager
def using_library(lib):
    """Route this module's calls to `lib` (for example the debug build) inside
    the block."""
    global _lib
    prev = load_library()
    _lib = lib
    try:
        yield lib
    finally:
        _lib = prev


def _check(code: int):
    if code != KDA_OK:
        raise KDAError(code, load_library().kda_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the KDA library must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the KDA library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_FP32
    raise ValueError(f"q/k/v must be bf16 or fp32, got {t.dtype}")


def make_desc(T: int, H: int, D: int, num_seqs: int, dtype_code: int, chunk: int = 64,
              ckpt_stride: int = 0, ckpt_capacity: int = 0, max_seq_len: int = 0,
              segment_chunks: int = 0, scalar_gate: bool = False, wait_limit: int = 0,
              recurrence_ctas: int = 0, conv_width: int = 0, conv_silu: bool = False) -> PrefillDesc:
    return PrefillDesc(num_seqs, T, H, D, D, dtype_code, chunk, ckpt_stride, ckpt_capacity,
                       max_seq_len, segment_chunks, int(bool(scalar_gate)), recurrence_ctas, conv_width,
                       int(bool(conv_silu)), wait_limit)


def workspace_size(desc: PrefillDesc) -> int:
    n = load_library().kda_prefill_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise KDAError(-1, load_library().kda_last_error().decode())
    return int(n)


def launch_count(desc: PrefillDesc) -> int:
    """Kernel launches one ``kda_prefill`` call with ``desc`` enqueues."""
    n = load_library().kda_prefill_launch_count(ctypes.byref(desc))
    if n < 0:
        raise KDAError(-1, load_library().kda_last_error().decode())
    return int(n)


def alloc_workspace(desc: PrefillDesc, device) -> torch.Tensor:
    return torch.empty(workspace_size(desc), dtype=torch.uint8, device=device)


def num_checkpoints(lens, ckpt_stride: int) -> int:
    return 0 if ckpt_stride <= 0 else int(sum(int(L) // ckpt_stride for L in lens))


def prefill(q, k, v, g, beta, init_state=None, cu_seqlens=None, *, num_seqs: Optional[int] = None,
            chunk: int = 64, ckpt_stride: int = 0, ckpts=None, ckpt_capacity: Optional[int] = None,
            out=None, final_state=None, workspace=None, stream=None, want_final: bool = True,
            max_seq_len: int = 0, segment_chunks: int = 0, wait_limit: int = 0, recurrence_ctas: int = 0):
    """Chunked KDA prefill through ``kda_prefill``.

    q, k: [T, H, D]; v: [T, H, D]; g: [T, H, D] (a decay per key channel) or
    [T, H] (one per head: the scalar-gate form); beta: [T, H]; init_state: [N, H, D, D] fp32 or
    None; cu_seqlens: [N + 1] int32 on the device, or None with ``num_seqs``
    equal-length sequences (default 1).  ``max_seq_len`` (0 = unknown) bounds
    every sequence's length; ``segment_chunks`` (0 = automatic) sets the
    overlap granularity of the tensor-core path.  Returns (out, final_state, ckpts).
    """
    T, H, D = q.shape
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    dev = q.device
    if out is None:
        out = torch.empty(T, H, v.shape[2], dtype=q.dtype, device=dev)
    if final_state is None and want_final:
        final_state = torch.empty(N, H, D, v.shape[2], dtype=torch.float32, device=dev)
    if ckpt_stride > 0 and ckpts is None:
        cap = ckpt_capacity if ckpt_capacity is not None else max(1, (T // ckpt_stride) + N)
        ckpts = torch.zeros(cap, H, D, v.shape[2], dtype=torch.float32, device=dev)
    cap = ckpt_capacity if ckpt_capacity is not None else (ckpts.shape[0] if ckpts is not None else 0)
    desc = make_desc(T, H, D, N, _dtype_code(q), chunk, ckpt_stride, cap, max_seq_len, segment_chunks,
                     scalar_gate=g.dim() == 2, wait_limit=wait_limit, recurrence_ctas=recurrence_ctas)
    if workspace is None:
        workspace = alloc_workspace(desc, dev)
    code = load_library().kda_prefill(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state), _ptr(cu_seqlens),
        _ptr(out), _ptr(final_state), _ptr(ckpts), ctypes.byref(desc), _ptr(workspace),
        ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(code)
    return out, final_state, ckpts


def prefill_noalloc(q, k, v, g, beta, init_state=None, cu_seqlens=None, *, num_seqs: Optional[int] = None,
                    chunk: int = 64, ckpt_stride: int = 0, ckpts=None, ckpt_capacity: Optional[int] = None,
                    out=None, final_state=None, stream=None, max_seq_len: int = 0,
                    segment_chunks: int = 0):
    """``kda_prefill_noalloc``: the same prefill with the library's built-in
    scratch array instead of a workspace, for callers that cannot allocate
    device memory.  Calls on one device share that array: do not let them
    overlap on the GPU.  Returns (out, final_state, ckpts)."""
    T, H, D = q.shape
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    dev = q.device
    if out is None:
        out = torch.empty(T, H, v.shape[2], dtype=q.dtype, device=dev)
    if final_state is None:
        final_state = torch.empty(N, H, D, v.shape[2], dtype=torch.float32, device=dev)
    if ckpt_stride > 0 and ckpts is None:
        cap = ckpt_capacity if ckpt_capacity is not None else max(1, (T // ckpt_stride) + N)
        ckpts = torch.zeros(cap, H, D, v.shape[2], dtype=torch.float32, device=dev)
    cap = ckpt_capacity if ckpt_capacity is not None else (ckpts.shape[0] if ckpts is not None else 0)
    desc = make_desc(T, H, D, N, _dtype_code(q), chunk, ckpt_stride, cap, max_seq_len, segment_chunks,
                     scalar_gate=g.dim() == 2)
    code = load_library().kda_prefill_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state), _ptr(cu_seqlens),
        _ptr(out), _ptr(final_state), _ptr(ckpts), ctypes.byref(desc), _stream(stream))
    _check(code)
    return out, final_state, ckpts


def prefill_fused(q, k, v, g, beta, init_state=None, cu_seqlens=None, *, conv_w=None, conv_silu: bool = False,
                  gate=None, conv_state_in=None, conv_state_out=None, num_seqs: Optional[int] = None,
                  chunk: int = 64, ckpt_stride: int = 0, ckpts=None, ckpt_capacity: Optional[int] = None, out=None,
                  final_state=None, workspace=None, stream=None, max_seq_len: int = 0, segment_chunks: int = 0):
    """``kda_prefill_fused``: the prefill with the short convolution of q, k, v
    (taps ``conv_w`` [3, W, H, D] fp32, W <= 4, optional SiLU; history
    ``conv_state_in`` [N, 3, W - 1, H, D] or None for zeros; the state after
    each sequence written to ``conv_state_out`` when given) before the
    recurrence and the output gate ``out = o * sigmoid(gate)`` (``gate``
    [T, H, Dv], the dtype of q) after it.  Returns (out, final_state, ckpts)."""
    T, H, D = q.shape
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    dev = q.device
    if out is None:
        out = torch.empty(T, H, v.shape[2], dtype=q.dtype, device=dev)
    if final_state is None:
        final_state = torch.empty(N, H, D, v.shape[2], dtype=torch.float32, device=dev)
    if ckpt_stride > 0 and ckpts is None:
        cap = ckpt_capacity if ckpt_capacity is not None else max(1, (T // ckpt_stride) + N)
        ckpts = torch.zeros(cap, H, D, v.shape[2], dtype=torch.float32, device=dev)
    cap = ckpt_capacity if ckpt_capacity is not None else (ckpts.shape[0] if ckpts is not None else 0)
    W = int(conv_w.shape[1]) if conv_w is not None else 0
    desc = make_desc(T, H, D, N, _dtype_code(q), chunk, ckpt_stride, cap, max_seq_len, segment_chunks,
                     scalar_gate=g.dim() == 2, conv_width=W, conv_silu=conv_silu)
    if workspace is None:
        workspace = alloc_workspace(desc, dev)
    code = load_library().kda_prefill_fused(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state), _ptr(cu_seqlens), _ptr(out),
        _ptr(final_state), _ptr(ckpts), _ptr(conv_w), _ptr(conv_state_in), _ptr(conv_state_out), _ptr(gate),
        ctypes.byref(desc), _ptr(workspace),
        ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(code)
    return out, final_state, ckpts


def prefill_pooled(q, k, v, g, beta, state_pool, init_slots=None, final_slots=None, cu_seqlens=None, *,
                   num_seqs: Optional[int] = None, chunk: int = 64, ckpt_stride: int = 0, ckpt_slots=None,
                   out=None, workspace=None, stream=None, max_seq_len: int = 0, segment_chunks: int = 0):
    """Chunked prefill through ``kda_prefill_pooled``: sequence n starts from
    slot ``init_slots[n]`` of ``state_pool`` [P, H, D, D] and its final state
    goes to slot ``final_slots[n]``; snapshot j goes to slot ``ckpt_slots[j]``
    (int32 tables on the device; None = none of that kind; an id outside
    [0, P) is skipped).  Returns out."""
    T, H, D = q.shape
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    dev = q.device
    if out is None:
        out = torch.empty(T, H, v.shape[2], dtype=q.dtype, device=dev)
    cap = ckpt_slots.numel() if (ckpt_stride > 0 and ckpt_slots is not None) else 0
    desc = make_desc(T, H, D, N, _dtype_code(q), chunk, ckpt_stride, cap, max_seq_len, segment_chunks,
                     scalar_gate=g.dim() == 2)
    if workspace is None:
        workspace = alloc_workspace(desc, dev)
    code = load_library().kda_prefill_pooled(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(out), _ptr(state_pool),
        ctypes.c_int64(state_pool.shape[0]), _ptr(init_slots), _ptr(final_slots),
        _ptr(ckpt_slots) if cap else None, ctypes.byref(desc), _ptr(workspace),
        ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(code)
    return out


def prefill_status(workspace: torch.Tensor, stream=None) -> int:
    """Device-side status of the last prefill on ``workspace`` (synchronises)."""
    return int(load_library().kda_prefill_status(_ptr(workspace), _stream(stream)))


def decode(q, k, v, g, beta, state, out=None, stream=None):
    """One decode step through ``kda_decode``; ``state`` [N, H, D, D] is updated in place."""
    N, H, D = q.shape
    if out is None:
        out = torch.empty(N, H, v.shape[2], dtype=q.dtype, device=q.device)
    code = load_library().kda_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                                     _ptr(out), N, H, D, v.shape[2], _dtype_code(q), _stream(stream))
    _check(code)
    return out


def decode_fused(q, k, v, g, beta, state, *, conv_w=None, conv_silu: bool = False, conv_state=None, gate=None,
                 out=None, stream=None):
    """One decode step through ``kda_decode_fused``: q, k, v [N, H, D]
    convolved with the history ``conv_state`` [N, 3, W - 1, H, D] (advanced in
    place; None: zeros), the step on ``state`` [N, H, D, D] (in place), the
    output gated by ``gate`` [N, H, D] (None: none)."""
    N, H, D = q.shape
    if out is None:
        out = torch.empty(N, H, v.shape[2], dtype=q.dtype, device=q.device)
    W = int(conv_w.shape[1]) if conv_w is not None else 0
    code = load_library().kda_decode_fused(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(conv_state), _ptr(conv_w), _ptr(gate),
        _ptr(out), N, H, D, v.shape[2], _dtype_code(q), W, int(bool(conv_silu)), _stream(stream))
    _check(code)
    return out


def decode_paged(q, k, v, g, beta, state_pool, slot_ids, out=None, stream=None, status=None):
    """One decode step through ``kda_decode_paged``: sequence n reads and
    updates slot ``slot_ids[n]`` of ``state_pool`` [P, H, D, D] (int32 ids on
    the device; an id outside [0, P) marks a padding row with a zero output).
    ``status`` (an int32 device tensor holding 0, or None) is set to
    KDA_ERR_INVALID_ARG when two sequences name the same slot."""
    N, H, D = q.shape
    if out is None:
        out = torch.empty(N, H, v.shape[2], dtype=q.dtype, device=q.device)
    code = load_library().kda_decode_paged(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_pool),
        ctypes.c_int64(state_pool.shape[0]), _ptr(slot_ids), _ptr(out), N, H, D, v.shape[2],
        _dtype_code(q), _ptr(status), _stream(stream))
    _check(code)
    return out


def decode_multi(q, k, v, g, beta, state, commit_len=None, slot_ids=None, out=None, stream=None,
                 status=None):
    """m tokens per sequence through ``kda_decode_multi``: q, k, g [N, m, H, D],
    v [N, m, H, D], beta [N, m, H]; ``state`` dense [N, H, D, D] or, with
    ``slot_ids``, a pool [P, H, D, D]; ``commit_len`` int32 [N] on the device
    (None: all m tokens) sets after how many tokens each state is written."""
    N, m, H, D = q.shape
    if out is None:
        out = torch.empty(N, m, H, v.shape[3], dtype=q.dtype, device=q.device)
    pool = state.shape[0] if slot_ids is not None else 0
    code = load_library().kda_decode_multi(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), ctypes.c_int64(pool),
        _ptr(slot_ids), _ptr(commit_len), _ptr(out), N, m, H, D, v.shape[3], _dtype_code(q), _ptr(status),
        _stream(stream))
    _check(code)
    return out


def _arg(name: str, t: Optional[torch.Tensor], shape, dtype, dev: int):
    """Address of an argument of the gated delta rule, the batch plan or the attention
    layers (None for None), after checking it: shape, type, device, contiguity."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on device {dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    if dev < 0:
        raise ValueError("tensors passed to the KDA library must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the KDA library must be contiguous")
    return t.data_ptr()


def _raw_stream(dev: int) -> int:
    """Handle of the current stream of device `dev` (a call of the binding spends
    more on the stream object than on its launch)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _new(shape, dtype, device, stream, zero: bool = False):
    """A tensor for a call on `stream` (None: the current one), allocated and
    cleared there: memory that another stream still uses is not handed out, and
    it goes back to that stream's calls."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _call(name: str, dev: int, stream, *args):
    """Calls the library's function `name` with `args` and the stream (the
    current one of device `dev` unless given), `dev` being the current device."""
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
    lib = _lib if _lib is not None else load_library()
    at = stream.cuda_stream if stream is not None else _raw_stream(dev)
    if dev == torch.cuda.current_device():
        code = getattr(lib, name)(*args, at)
    else:
        with torch.cuda.device(dev):
            code = getattr(lib, name)(*args, at)
    if code != KDA_OK:
        raise KDAError(code, lib.kda_last_error().decode())


def _gdn_tokens(q, k, v, g, beta, rows, out, stream):
    """Checks the token tensors (leading dims `rows`); returns (Hk, Hv, Dk, Dv,
    dtype code, out, device index, addresses of q, k, v, g, beta, out)."""
    r = len(rows)
    if q.dim() != r + 2 or v.dim() != r + 2:
        raise ValueError(f"q and v must have {r + 2} dims, got {q.dim()} and {v.dim()}")
    dt, dev = q.dtype, q.get_device()
    code = _dtype_code(q)
    Hk, Dk = q.shape[r:]
    Hv, Dv = v.shape[r:]
    per_qk, per_v, per_head = (*rows, Hk, Dk), (*rows, Hv, Dv), (*rows, Hv)
    tokens = (_arg("q", q, per_qk, dt, dev), _arg("k", k, per_qk, dt, dev), _arg("v", v, per_v, dt, dev),
              _arg("g", g, per_head, torch.float32, dev), _arg("beta", beta, per_head, torch.float32, dev))
    if out is None:
        out = _new(per_v, dt, q.device, stream)
        return (Hk, Hv, Dk, Dv, code, out, dev, tokens, out.data_ptr())
    return (Hk, Hv, Dk, Dv, code, out, dev, tokens, _arg("out", out, per_v, dt, dev))


def _gdn_workspace(desc, workspace, device, stream):
    """(workspace, its address, its bytes), allocated if None."""
    if workspace is not None:
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, the tensors on {device}")
        return workspace, _ptr(workspace), workspace.numel() * workspace.element_size()
    n = gdn_workspace_size(desc)
    workspace = _new((n,), torch.uint8, device, stream)
    return workspace, workspace.data_ptr(), n


def _gdn_longest(T: int, N: int, cu_seqlens, hint: int) -> int:
    """Upper bound of the sequences' lengths: the hint, else what equal sequences
    have, else 0 (unknown: the lengths are on the device)."""
    return hint if hint or cu_seqlens is not None else T // max(N, 1)


def make_gdn_desc(T: int, Hk: int, Hv: int, Dk: int, Dv: int, num_seqs: int, dtype_code: int, ckpt_stride: int = 0,
                  ckpt_capacity: int = 0, max_seq_len: int = 0, wait_limit: int = 0) -> GdnDesc:
    return GdnDesc(num_seqs, T, Hk, Hv, Dk, Dv, dtype_code, ckpt_stride, ckpt_capacity, max_seq_len, wait_limit)


def gdn_workspace_size(desc: GdnDesc) -> int:
    n = load_library().kda_gdn_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise KDAError(-1, load_library().kda_last_error().decode())
    return int(n)


def gdn_prefill(q, k, v, g, beta, init_state=None, cu_seqlens=None, *, num_seqs: Optional[int] = None,
                ckpt_stride: int = 0, ckpts=None, ckpt_capacity: Optional[int] = None, out=None, final_state=None,
                workspace=None, stream=None, want_final: bool = True, max_seq_len: int = 0, wait_limit: int = 0):
    """Prefill of the gated delta rule through ``kda_gdn_prefill``: one decay
    per token and value head, value heads sharing a query/key head.

    q, k: [T, Hk, Dk]; v: [T, Hv, Dv] (Hv a multiple of Hk; Dk 64 or 128, Dv a
    multiple of 64); g, beta: [T, Hv] fp32; init_state: [N, Hv, Dk, Dv] fp32 or
    None; cu_seqlens: [N + 1] int32 on the device (its last entry may be below
    T: the rows behind are padding and their outputs are left as they were), or
    None with ``num_seqs`` equal sequences.  A caller's ``workspace`` is sized by
    ``gdn_workspace_size`` of a desc with the same ``max_seq_len``, which without
    offsets is T // num_seqs unless given.  Returns (out, final_state, ckpts).
    """
    T, f32 = q.shape[0], torch.float32
    Hk, Hv, Dk, Dv, code, out, dev, tokens, out_at = _gdn_tokens(q, k, v, g, beta, (T,), out, stream)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    if final_state is None and want_final:
        final_state = _new((N, Hv, Dk, Dv), f32, q.device, stream)
    if ckpt_stride > 0 and ckpts is None:
        cap = ckpt_capacity if ckpt_capacity is not None else max(1, T // ckpt_stride)
        ckpts = _new((cap, Hv, Dk, Dv), f32, q.device, stream, zero=True)
    cap = ckpts.shape[0] if ckpts is not None else 0
    if ckpt_capacity is not None and ckpt_capacity > cap:
        raise ValueError(f"ckpt_capacity {ckpt_capacity} > {cap} blocks of ckpts")
    desc = make_gdn_desc(T, Hk, Hv, Dk, Dv, N, code, ckpt_stride, cap if ckpt_capacity is None else ckpt_capacity,
                         _gdn_longest(T, N, cu_seqlens, max_seq_len), wait_limit)
    state = (N, Hv, Dk, Dv)
    args = (*tokens, _arg("init_state", init_state, state, f32, dev),
            _arg("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev), out_at,
            _arg("final_state", final_state, state, f32, dev), _arg("ckpts", ckpts, (cap, Hv, Dk, Dv), f32, dev))
    workspace, ws_at, ws_bytes = _gdn_workspace(desc, workspace, q.device, stream)
    _call("kda_gdn_prefill", dev, stream, *args, ctypes.byref(desc), ws_at, ws_bytes)
    return out, final_state, ckpts


def gdn_prefill_pooled(q, k, v, g, beta, state_pool, init_slots=None, final_slots=None, cu_seqlens=None, *,
                       num_seqs: Optional[int] = None, ckpt_stride: int = 0, ckpt_slots=None, out=None,
                       workspace=None, stream=None, max_seq_len: int = 0, wait_limit: int = 0):
    """``gdn_prefill`` with its states in slots of ``state_pool`` [P, Hv, Dk, Dv]
    (``kda_gdn_prefill_pooled``): int32 tables on the device, as in
    ``prefill_pooled`` and as ``plan_batch`` builds them.  Returns out."""
    T, i32 = q.shape[0], torch.int32
    Hk, Hv, Dk, Dv, code, out, dev, tokens, out_at = _gdn_tokens(q, k, v, g, beta, (T,), out, stream)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    P = state_pool.shape[0]
    cap = ckpt_slots.numel() if (ckpt_stride > 0 and ckpt_slots is not None) else 0
    desc = make_gdn_desc(T, Hk, Hv, Dk, Dv, N, code, ckpt_stride, cap, _gdn_longest(T, N, cu_seqlens, max_seq_len),
                         wait_limit)
    args = (*tokens, _arg("cu_seqlens", cu_seqlens, (N + 1,), i32, dev), out_at,
            _arg("state_pool", state_pool, (P, Hv, Dk, Dv), torch.float32, dev), P,
            _arg("init_slots", init_slots, (N,), i32, dev), _arg("final_slots", final_slots, (N,), i32, dev),
            _arg("ckpt_slots", ckpt_slots, (cap,), i32, dev) if cap else None)
    workspace, ws_at, ws_bytes = _gdn_workspace(desc, workspace, q.device, stream)
    _call("kda_gdn_prefill_pooled", dev, stream, *args, ctypes.byref(desc), ws_at, ws_bytes)
    return out


def _status_arg(status, dev):
    return _arg("status", status, (1,) if status is not None and status.dim() else (), torch.int32, dev)


def gdn_decode(q, k, v, g, beta, state, slot_ids=None, out=None, stream=None, status=None):
    """One decode step of the gated delta rule through ``kda_gdn_decode``: q, k
    [N, Hk, Dk], v [N, Hv, Dv], g, beta [N, Hv]; ``state`` [N, Hv, Dk, Dv] or,
    with ``slot_ids`` (int32 [N], an id outside [0, P) marks a padding row), a
    pool [P, Hv, Dk, Dv], updated in place.  ``status`` as in ``decode_paged``."""
    N = q.shape[0]
    Hk, Hv, Dk, Dv, code, out, dev, tokens, out_at = _gdn_tokens(q, k, v, g, beta, (N,), out, stream)
    P = N if slot_ids is None else state.shape[0]
    _call("kda_gdn_decode", dev, stream, *tokens, _arg("state", state, (P, Hv, Dk, Dv), torch.float32, dev), P,
          _arg("slot_ids", slot_ids, (N,), torch.int32, dev), out_at, N, Hk, Hv, Dk, Dv, code,
          _status_arg(status, dev))
    return out


def gdn_decode_multi(q, k, v, g, beta, state, commit_len=None, slot_ids=None, out=None, stream=None, status=None):
    """m tokens per sequence through ``kda_gdn_decode_multi``: q, k
    [N, m, Hk, Dk], v [N, m, Hv, Dv], g, beta [N, m, Hv]; ``commit_len`` int32
    [N] (None: all m tokens) sets after how many tokens each state is written."""
    N, m = q.shape[:2]
    Hk, Hv, Dk, Dv, code, out, dev, tokens, out_at = _gdn_tokens(q, k, v, g, beta, (N, m), out, stream)
    P = N if slot_ids is None else state.shape[0]
    _call("kda_gdn_decode_multi", dev, stream, *tokens, _arg("state", state, (P, Hv, Dk, Dv), torch.float32, dev), P,
          _arg("slot_ids", slot_ids, (N,), torch.int32, dev), _arg("commit_len", commit_len, (N,), torch.int32, dev),
          out_at, N, m, Hk, Hv, Dk, Dv, code, _status_arg(status, dev))
    return out


def plan_batch(lens, state_slots, *, total_tokens: int, past=None, resume_slots=None, ckpt_stride: int = 0,
               ckpt_capacity: int = 0, free_slots=None, free_head=None, snap_table=None, out: Optional[BatchPlan] = None,
               status=None, stream=None) -> BatchPlan:
    """The batch's offsets, slot tables and token maps, built on the device from
    request lengths (``kda_plan_batch``); every table is int32.

    lens, state_slots, past, resume_slots: [N]; free_slots: [F] (None: none);
    free_head: [1] first unused entry of free_slots (None: 0); snap_table:
    [N, cols], entered in place.  The plan's state_slots are the final_slots of a
    prefill; as slot_ids of a decode step, put -1 for requests without a token, and
    prefill new requests first (a slot just taken holds no state).  ``out``: a
    BatchPlan to write to (its state_slots and free_head may be the inputs
    themselves).  ``status``: an
    int32 tensor of one value, set to 0 or an error code.
    """
    N, dev, i32 = lens.numel(), lens.get_device(), torch.int32
    F = 0 if free_slots is None else free_slots.numel()
    cols = 0 if snap_table is None else snap_table.shape[-1]
    sizes = (N + 1, N, N, N + 1, ckpt_capacity, total_tokens, total_tokens, 1)
    if free_head is None:
        free_head = _new((1,), i32, lens.device, stream, zero=True)
    tables = [_arg(name, t, (N,), i32, dev) for name, t in (("lens", lens), ("past", past), ("resume_slots", resume_slots),
                                                            ("state_slots", state_slots))]
    if out is None:   # one allocation; its parts need no check (nor, as integers, autograd's views)
        whole = _new((sum(sizes),), i32, lens.device, stream)
        out = BatchPlan(*whole.unsafe_split_with_sizes(sizes))
        base = whole.data_ptr()
        outs = [base] + [base + 4 * end for end in accumulate(sizes[:-1])]
    else:
        outs = [_arg(name, t, (n,), i32, dev) for name, t, n in zip(BatchPlan._fields, out, sizes)]
    _call("kda_plan_batch", dev, stream, *tables, _arg("free_slots", free_slots, (F,), i32, dev), F,
          _arg("free_head", free_head, (1,), i32, dev), N, total_tokens, ckpt_stride, ckpt_capacity,
          _arg("snap_table", snap_table, (N, cols), i32, dev), cols, *outs, _status_arg(status, dev))
    return out


# ---------------------------------------------------------------- attention layers
def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(inv_freq [rotary_dim / 2] fp32, rope_scale) for ``kv_append``, formed in 64 bits.

    Pair i turns by base^(-2i / rotary_dim) a position.  For contexts ``factor`` times the ``original_len`` that a
    model was trained on: ``scaling`` "linear" divides every frequency by factor; "base" raises the base until the
    slowest pair is factor times slower; "parts" divides the pairs that turn less than beta_slow times in original_len,
    keeps those that turn more than beta_fast times, and between them weighs kept and divided linearly in the logarithm of the
    turns (that is, in the number of the pair, without rounding the ends to whole pairs); rope_scale is 0.1 ln(factor) + 1.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not base > 1 or not factor >= 1:
        raise ValueError(f"base must be above 1 and factor at least 1, got {base} and {factor}")
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError("scaling by the base needs two pairs")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = float(base) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original_len < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("scaling by parts needs original_len >= 1 and beta_fast > beta_slow > 0")
        turns = original_len * f / (2 * math.pi)
        keep = ((turns / beta_slow).log() / math.log(beta_fast / beta_slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
    return f.to(torch.float32).to(device), scale


def _heads_arg(name: str, t, heads: int, T: int, D: int, dtype, dev: int):
    """(address, token stride) of [T, heads, D] whose heads are contiguous within a token (a part of a wider row)."""
    if t is None:
        return None, 0
    if t.shape != (T, heads, D) or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} {[T, heads, D]} on device {dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    if dev < 0:
        raise ValueError("tensors passed to the KDA library must live on a CUDA device")
    by_token, by_head, by_dim = t.stride()
    if by_dim != 1 or (heads > 1 and by_head != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {t.stride()}")
    if T <= 1:
        return t.data_ptr(), heads * D
    if by_token < heads * D:
        raise ValueError(f"{name}: tokens may not overlap, got strides {t.stride()}")
    return t.data_ptr(), by_token


def _kv_dtype(q_dtype, cache) -> int:
    if cache.dtype is torch.float8_e4m3fn:
        return DTYPE_E4M3
    if cache.dtype is not q_dtype:
        raise ValueError(f"the cache must be {q_dtype} or float8_e4m3fn, got {cache.dtype}")
    return _dtype_code(cache)


def _cache_args(k_cache, v_cache, k_scale, v_scale, Hkv: int, D: int, dev: int):
    """(addresses of the cache and its scales, pages, page size)."""
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be [pages, Hkv, page, D], got {list(k_cache.shape)}")
    pages, _, page, _ = k_cache.shape
    shape = (pages, Hkv, page, D)
    return (_arg("k_cache", k_cache, shape, k_cache.dtype, dev), _arg("v_cache", v_cache, shape, k_cache.dtype, dev),
            _arg("k_scale", k_scale, shape[:3], torch.float32, dev), _arg("v_scale", v_scale, shape[:3], torch.float32, dev),
            pages, page)


def kv_append(q, k, v, positions, *, seq_ids=None, page_table=None, k_cache=None, v_cache=None, k_scale=None, v_scale=None,
              inv_freq=None, interleaved: bool = False, rope_scale: float = 1.0, q_out=None, k_out=None,
              want_k: Optional[bool] = None, status=None, stream=None):
    """Rotates new tokens' queries and keys and writes keys and values into a paged cache (``kda_kv_append``).

    q: [T, Hq, D] or None; k, v: [T, Hkv, D], rows possibly parts of wider ones (the output of one projection); positions,
    seq_ids: int32 [T] (``plan_batch``'s; negative: a padding row, left as it is); k_cache, v_cache: [pages, Hkv, page, D]
    of q's type, or float8_e4m3fn with k_scale, v_scale [pages, Hkv, page] fp32; page_table: int32 [N, cols]; without
    them only q and k are rotated (v may be None).  inv_freq: fp32 [R / 2] (``rope_frequencies``; None: no rotation).
    q_out, k_out may be q, k; ``want_k``: whether k_out is written (None: only without a cache, or if k_out is given).
    ``status`` as in ``decode_paged``, set where a row has no page.  Returns (q_out, k_out).
    """
    if k_cache is None and any(x is not None for x in (page_table, v_cache, k_scale, v_scale)):
        raise ValueError("page_table, v_cache, k_scale and v_scale go with k_cache")
    T, Hkv, D = k.shape
    dt, dev, i32 = k.dtype, k.get_device(), torch.int32
    code = _dtype_code(k)
    Hq = q.shape[1] if q is not None else Hkv
    q_at, q_step = _heads_arg("q", q, Hq, T, D, dt, dev)
    k_at, k_step = _heads_arg("k", k, Hkv, T, D, dt, dev)
    v_at, v_step = _heads_arg("v", v, Hkv, T, D, dt, dev)
    if q is not None and q_out is None:
        q_out = _new((T, Hq, D), dt, k.device, stream)
    if k_out is None and (want_k if want_k is not None else k_cache is None):
        k_out = _new((T, Hkv, D), dt, k.device, stream)
    N, cols, pages, page, kv = 0, 0, 0, 0, code
    cache = (None, None, None, None)
    if k_cache is not None:
        if page_table is None or page_table.dim() != 2 or v_cache is None or v is None or seq_ids is None:
            raise ValueError("a cache needs page_table [N, cols], v_cache, v and seq_ids")
        kv = _kv_dtype(dt, k_cache)
        *cache, pages, page = _cache_args(k_cache, v_cache, k_scale, v_scale, Hkv, D, dev)
        N, cols = page_table.shape
    R = 2 * inv_freq.numel() if inv_freq is not None else 0
    desc = AppendDesc(T, Hq, Hkv, D, code, kv, R, int(bool(interleaved)), rope_scale, N, page, cols, pages, q_step, k_step, v_step)
    _call("kda_kv_append", dev, stream, q_at, k_at, v_at, _arg("positions", positions, (T,), i32, dev),
          _arg("seq_ids", seq_ids, (T,), i32, dev), _arg("page_table", page_table, (N, cols), i32, dev),
          _arg("inv_freq", inv_freq, (R // 2,), torch.float32, dev), _arg("q_out", q_out, (T, Hq, D), dt, dev),
          _arg("k_out", k_out, (T, Hkv, D), dt, dev), *cache, _status_arg(status, dev), ctypes.byref(desc))
    return q_out, k_out


def make_attn_desc(T: int, Hq: int, Hkv: int, D: int, num_seqs: int, dtype_code: int, kv_dtype: Optional[int] = None,
                   page_size: int = 0, pages_per_seq: int = 0, num_pages: int = 0, max_seq_len: int = 0, scale: float = 0.0,
                   wait_limit: int = 0) -> AttnDesc:
    return AttnDesc(num_seqs, T, Hq, Hkv, D, dtype_code, dtype_code if kv_dtype is None else kv_dtype, page_size, pages_per_seq,
                    num_pages, max_seq_len, scale, wait_limit)


def attn_workspace_size(desc: AttnDesc, decode: bool = False) -> int:
    """Bytes of a prefill's workspace, or of a decode call's."""
    lib = _lib if _lib is not None else load_library()
    n = (lib.kda_attn_decode_workspace_size if decode else lib.kda_attn_workspace_size)(ctypes.byref(desc))
    if n == 0:
        raise KDAError(-1, load_library().kda_last_error().decode())
    return int(n)


def _scale_arg(scale: Optional[float]) -> float:
    """The desc's scale (0: the default)."""
    if scale is None:
        return 0.0
    if not 0 < ctypes.c_float(scale).value < math.inf:
        raise ValueError(f"scale must be None, or positive and finite in fp32, got {scale}")
    return scale


def _attn_outputs(q, out, lse, want_lse, dev, stream):
    """(out, lse, their addresses), allocated if None (lse only if wanted)."""
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q.shape, q.dtype, q.device, stream)
        out_at = out.data_ptr()
    else:
        out_at = _arg("out", out, q.shape, q.dtype, dev)
    if lse is None and want_lse:
        lse = _new(q.shape[:-1], torch.float32, q.device, stream)
        return out, lse, out_at, lse.data_ptr()
    return out, lse, out_at, _arg("lse", lse, q.shape[:-1], torch.float32, dev)


def _attn_workspace(desc, workspace, device, stream, decode=False):
    """(workspace, its address, its bytes), allocated if None."""
    if workspace is not None:
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, the tensors on {device}")
        return workspace, _ptr(workspace), workspace.numel() * workspace.element_size()
    n = attn_workspace_size(desc, decode)
    workspace = _new((n,), torch.uint8, device, stream)
    return workspace, workspace.data_ptr(), n


def attn_prefill(q, k, v, cu_seqlens=None, *, num_seqs: Optional[int] = None, scale: Optional[float] = None, out=None, lse=None,
                 want_lse: bool = False, workspace=None, stream=None, max_seq_len: int = 0, wait_limit: int = 0):
    """Causal attention of packed prompts through ``kda_attn_prefill``: q [T, Hq, D], k, v [T, Hkv, D] (Hq a multiple of
    Hkv, D 64 or 128, bf16 or fp32), cu_seqlens as in ``gdn_prefill``; scale None: D ** -0.5.  Returns (out, lse), lse
    [T, Hq] fp32 or None."""
    T, Hq, D = q.shape
    Hkv, dt, dev = k.shape[1], q.dtype, q.get_device()
    code = _dtype_code(q)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (num_seqs or 1)
    ins = (_arg("q", q, (T, Hq, D), dt, dev), _arg("k", k, (T, Hkv, D), dt, dev), _arg("v", v, (T, Hkv, D), dt, dev),
           _arg("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev))
    out, lse, *outs = _attn_outputs(q, out, lse, want_lse, dev, stream)
    desc = make_attn_desc(T, Hq, Hkv, D, N, code, max_seq_len=_gdn_longest(T, N, cu_seqlens, max_seq_len), scale=_scale_arg(scale),
                          wait_limit=wait_limit)
    workspace, ws_at, ws_bytes = _attn_workspace(desc, workspace, q.device, stream)
    _call("kda_attn_prefill", dev, stream, *ins, *outs, ctypes.byref(desc), ws_at, ws_bytes)
    return out, lse


def _paged_args(q, k_cache, v_cache, page_table, kv_lens, k_scale, v_scale):
    """(Hq, Hkv, D, N, cache arguments, keyword arguments of the desc)."""
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [N, cols], got {list(page_table.shape)}")
    Hq, D = q.shape[-2:]
    dev = q.get_device()
    Hkv = k_cache.shape[1] if k_cache.dim() == 4 else 0
    *cache, pages, page = _cache_args(k_cache, v_cache, k_scale, v_scale, Hkv, D, dev)
    N, cols = page_table.shape
    tables = (_arg("page_table", page_table, (N, cols), torch.int32, dev), _arg("kv_lens", kv_lens, (N,), torch.int32, dev))
    return Hq, Hkv, D, N, (*cache, *tables), dict(kv_dtype=_kv_dtype(q.dtype, k_cache), page_size=page, pages_per_seq=cols,
                                                  num_pages=pages)


def attn_prefill_paged(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens=None, *, k_scale=None, v_scale=None,
                       scale: Optional[float] = None, out=None, lse=None, want_lse: bool = False, workspace=None, stream=None,
                       max_seq_len: int = 0, wait_limit: int = 0):
    """``attn_prefill`` over a paged cache (``kda_attn_prefill_paged``): the queries q [T, Hq, D] of sequence n are the last
    tokens of its kv_lens[n] (int32 [N], the new ones included); the cache as ``kv_append`` writes it.  Returns (out, lse)."""
    T, dev = q.shape[0], q.get_device()
    code = _dtype_code(q)
    Hq, Hkv, D, N, cache, kw = _paged_args(q, k_cache, v_cache, page_table, kv_lens, k_scale, v_scale)
    ins = (_arg("q", q, (T, Hq, D), q.dtype, dev), _arg("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev))
    out, lse, *outs = _attn_outputs(q, out, lse, want_lse, dev, stream)
    desc = make_attn_desc(T, Hq, Hkv, D, N, code, max_seq_len=_gdn_longest(T, N, cu_seqlens, max_seq_len), scale=_scale_arg(scale),
                          wait_limit=wait_limit, **kw)
    workspace, ws_at, ws_bytes = _attn_workspace(desc, workspace, q.device, stream)
    _call("kda_attn_prefill_paged", dev, stream, *ins, *cache, *outs, ctypes.byref(desc), ws_at, ws_bytes)
    return out, lse


def _attn_decode(q, m, k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, scale, out, lse, want_lse, status, workspace,
                 stream):
    dev = q.get_device()
    code = _dtype_code(q)
    Hq, Hkv, D, N, cache, kw = _paged_args(q, k_cache, v_cache, page_table, kv_lens, k_scale, v_scale)
    shape = (N, Hq, D) if m is None else (N, m, Hq, D)
    q_at = _arg("q", q, shape, q.dtype, dev)
    out, lse, *outs = _attn_outputs(q, out, lse, want_lse, dev, stream)
    if N == 0:
        return out, lse
    desc = make_attn_desc(N * (1 if m is None else m), Hq, Hkv, D, N, code, scale=_scale_arg(scale), **kw)
    workspace, ws_at, ws_bytes = _attn_workspace(desc, workspace, q.device, stream, decode=True)
    _call("kda_attn_decode", dev, stream, q_at, *cache, *outs, ctypes.byref(desc), _status_arg(status, dev), ws_at, ws_bytes)
    return out, lse


def attn_decode(q, k_cache, v_cache, page_table, kv_lens, *, k_scale=None, v_scale=None, scale: Optional[float] = None,
                out=None, lse=None, want_lse: bool = False, status=None, workspace=None, stream=None):
    """Attention of one new token a sequence over a paged cache (``kda_attn_decode``): q [N, Hq, D], the token being the
    last of kv_lens[n] (0: zeros).  ``status`` as in ``decode_paged``, set for lengths and pages out of range.  Returns
    (out, lse), lse [N, Hq] fp32 or None."""
    return _attn_decode(q, None, k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, scale, out, lse, want_lse, status,
                        workspace, stream)


def attn_decode_multi(q, k_cache, v_cache, page_table, kv_lens, *, k_scale=None, v_scale=None, scale: Optional[float] = None,
                      out=None, lse=None, want_lse: bool = False, status=None, workspace=None, stream=None):
    """``attn_decode`` of m new tokens a sequence (drafted tokens to verify): q [N, m, Hq, D], token i at position
    kv_lens[n] - m + i and seeing no later one."""
    return _attn_decode(q, q.shape[1], k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, scale, out, lse, want_lse,
                        status, workspace, stream)
