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
DTYPE_BF16, DTYPE_FP32 = 0, 1

# Every symbol include/kda.h declares.
EXPORTS = ("kda_prefill_workspace_size", "kda_prefill_launch_count", "kda_prefill", "kda_prefill_status",
           "kda_prefill_pooled", "kda_prefill_fused", "kda_decode", "kda_decode_fused", "kda_decode_paged",
           "kda_decode_multi", "kda_prefill_noalloc", "kda_gdn_workspace_size", "kda_gdn_prefill",
           "kda_gdn_prefill_pooled", "kda_gdn_decode", "kda_gdn_decode_multi", "kda_plan_batch", "kda_last_error",
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
    """Address of an argument of the gated delta rule or of the batch plan (None
    for None), after checking it: shape, type, device, contiguity."""
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
