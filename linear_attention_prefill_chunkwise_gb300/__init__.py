"""GB300 (sm_103a) Lightning Attention chunkwise prefill and speculative-decoding ops, and the
gated linear recurrence, the RMS norm and a hybrid model's softmax attention beside them.

``la_prefill_fwd`` (include/la_prefill.h), ``la_prefill_bwd`` (include/la_backward.h),
``la_prefill_fwd_segmented``,
``la_prefill_fwd_segmented_static`` and ``la_prefill_segmented_workspace``
(include/la_segment.h) and ``la_decode_mtp``,
``la_verify``, ``la_commit`` (include/la_decode.h), ``la_gated_scan_fwd``, ``la_gated_scan_bwd``,
``la_gated_decode``, ``la_gated_verify``, ``la_gated_commit`` (include/la_gated.h),
``la_rms_norm_fwd``, ``la_rms_norm_fwd_fp8``, ``la_rms_norm_bwd`` (include/la_norm.h),
``la_qk_norm_rope_fwd``, ``la_qk_norm_rope_bwd`` (include/la_rotary.h) and ``la_attn_prefill_fwd``,
``la_attn_prefill_bwd``, ``la_attn_verify``, ``la_attn_commit`` (include/la_attention.h) are thin ctypes bindings of the C
entry points of the same names: they check dtypes and shapes of torch tensors, pass their device
pointers and the current CUDA stream, and raise on a non-OK status.  Every step of the
computation runs in the library's CUDA kernels; there is no other implementation in
this package and no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

from . import build as _build

__all__ = ["la_prefill_fwd", "la_prefill_fwd_segmented", "la_prefill_fwd_segmented_static", "la_prefill_bwd",
           "la_prefill_bwd_workspace", "la_prefill_fwd_d256", "la_prefill_d256_workspace",
           "la_prefill_fwd_d256_segmented", "la_prefill_d256_segmented_workspace",
           "la_prefill_segmented_workspace", "la_decode_mtp", "la_verify", "la_commit",
           "la_gated_scan_fwd", "la_gated_scan_bwd", "la_gated_scan_workspace", "la_gated_decode", "la_gated_verify",
           "la_gated_commit", "la_rms_norm_fwd", "la_rms_norm_fwd_fp8", "la_rms_norm_bwd", "la_rms_norm_bwd_workspace",
           "la_qk_norm_rope_fwd", "la_qk_norm_rope_bwd", "la_qk_norm_rope_bwd_workspace", "la_attn_prefill_fwd",
           "la_attn_prefill_bwd", "la_attn_prefill_bwd_workspace", "la_attn_verify", "la_attn_verify_workspace",
           "la_attn_commit",
           "LaError", "load_library", "SCHEDULES", "DEV_ERR_BAD_SEQLENS",
           "DEV_ERR_BAD_INDEX", "DEV_ERR_TIMEOUT", "EXPORTED_SYMBOLS"]

SCHEDULES = {"auto": 0, "persistent": 1, "non_persistent": 2}
DEV_ERR_BAD_SEQLENS = 1
DEV_ERR_BAD_INDEX = 2
DEV_ERR_TIMEOUT = 4
EXPORTED_SYMBOLS = ("la_prefill_fwd", "la_status_string", "la_last_error", "la_prefill_smem_bytes",
                    "la_decode_mtp", "la_verify",
                    "la_commit", "la_prefill_segmented_workspace", "la_prefill_fwd_segmented",
                    "la_prefill_fwd_segmented_static", "la_prefill_bwd_workspace", "la_prefill_bwd",
                    "la_prefill_d256_workspace", "la_prefill_fwd_d256", "la_prefill_d256_segmented_workspace",
                    "la_prefill_fwd_d256_segmented", "la_gated_scan_workspace", "la_gated_scan_fwd", "la_gated_scan_bwd",
                    "la_gated_decode", "la_gated_verify", "la_gated_commit", "la_rms_norm_fwd", "la_rms_norm_fwd_fp8",
                    "la_rms_norm_bwd_workspace", "la_rms_norm_bwd", "la_qk_norm_rope_fwd",
                    "la_qk_norm_rope_bwd_workspace", "la_qk_norm_rope_bwd", "la_attn_prefill_fwd",
                    "la_attn_prefill_bwd_workspace", "la_attn_prefill_bwd", "la_attn_verify_workspace", "la_attn_verify",
                    "la_attn_commit")

_lock = threading.Lock()
_lib = None


class LaError(RuntimeError):
    """A non-OK la_status returned by the C library."""

    def __init__(self, status: int, name: str, detail: str):
        super().__init__(f"{name}: {detail}")
        self.status = status
        self.name = name


def load_library(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libla_prefill.so (building it first when it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if build_if_missing:
                path = _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library not built: {path} (run linear_attention_prefill_chunkwise_gb300.build)")
            lib = ctypes.CDLL(path)
            vp, i32p, fp = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
            lib.la_prefill_fwd.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, i32p, i32p, vp, fp] + \
                [ctypes.c_int] * 8 + [ctypes.c_int, vp, vp]
            lib.la_prefill_fwd.restype = ctypes.c_int
            lib.la_status_string.argtypes = [ctypes.c_int]
            lib.la_status_string.restype = ctypes.c_char_p
            lib.la_last_error.argtypes = []
            lib.la_last_error.restype = ctypes.c_char_p
            lib.la_prefill_smem_bytes.argtypes = []
            lib.la_prefill_smem_bytes.restype = ctypes.c_int
            ints = [ctypes.c_int] * 7  # B, T, H, HV, D, V, pool_size
            lib.la_decode_mtp.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, i32p, vp] + ints + [vp, vp]
            lib.la_decode_mtp.restype = ctypes.c_int
            lib.la_verify.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, i32p, vp, vp, vp] + ints + [vp, vp]
            lib.la_verify.restype = ctypes.c_int
            lib.la_commit.argtypes = [fp, i32p, vp, vp, i32p, fp] + ints + [vp, vp]
            lib.la_commit.restype = ctypes.c_int
            lib.la_prefill_segmented_workspace.argtypes = [ctypes.c_int] * 6 + [vp, vp]
            lib.la_prefill_segmented_workspace.restype = ctypes.c_int
            lib.la_prefill_fwd_segmented.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, i32p, i32p, vp, fp] + \
                [ctypes.c_int] * 9 + [vp, ctypes.c_size_t, vp, vp]
            lib.la_prefill_fwd_segmented.restype = ctypes.c_int
            lib.la_prefill_fwd_segmented_static.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, i32p, i32p, vp,
                                                            fp] + [ctypes.c_int] * 9 + [vp, vp]
            lib.la_prefill_fwd_segmented_static.restype = ctypes.c_int
            lib.la_prefill_bwd_workspace.argtypes = [ctypes.c_int] * 8 + [vp]
            lib.la_prefill_bwd_workspace.restype = ctypes.c_int
            lib.la_prefill_bwd.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, vp, fp, i32p, i32p, vp, vp, vp, fp] + \
                [ctypes.c_int] * 8 + [vp, ctypes.c_size_t, vp, vp]
            lib.la_prefill_bwd.restype = ctypes.c_int
            lib.la_prefill_d256_workspace.argtypes = [ctypes.c_int] * 5 + [vp]
            lib.la_prefill_d256_workspace.restype = ctypes.c_int
            lib.la_prefill_fwd_d256.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, i32p, i32p, vp, fp] + \
                [ctypes.c_int] * 8 + [vp, ctypes.c_size_t, vp, vp]
            lib.la_prefill_fwd_d256.restype = ctypes.c_int
            lib.la_prefill_d256_segmented_workspace.argtypes = [ctypes.c_int] * 7 + [vp, vp]
            lib.la_prefill_d256_segmented_workspace.restype = ctypes.c_int
            lib.la_prefill_fwd_d256_segmented.argtypes = [vp, vp, vp, fp, ctypes.c_float, fp, i32p, i32p, vp, fp] + \
                [ctypes.c_int] * 9 + [vp, ctypes.c_size_t, vp, vp]
            lib.la_prefill_fwd_d256_segmented.restype = ctypes.c_int
            i64, i32 = ctypes.c_int64, ctypes.c_int
            lib.la_gated_scan_workspace.argtypes = [i32] * 7 + [vp]
            lib.la_gated_scan_fwd.argtypes = [vp] * 9 + [i64] * 4 + [i32] * 6 + [vp, ctypes.c_size_t, vp, vp]
            lib.la_gated_scan_bwd.argtypes = [vp] * 15 + [i64] * 8 + [i32] * 6 + [vp, ctypes.c_size_t, vp, vp]
            lib.la_gated_decode.argtypes = [vp] * 7 + [i64] * 4 + [i32] * 5 + [vp, vp]
            lib.la_gated_verify.argtypes = [vp] * 7 + [i64] * 4 + [i32] * 5 + [vp, vp]
            lib.la_gated_commit.argtypes = [vp] * 7 + [i64] * 3 + [i32] * 5 + [vp, vp]
            lib.la_rms_norm_fwd.argtypes = [vp] * 3 + [ctypes.c_float] + [vp] * 2 + [i64] * 4 + [i32] * 3 + [vp] * 2
            lib.la_rms_norm_fwd_fp8.argtypes = [vp] * 3 + [ctypes.c_float] + [vp] * 3 + [i64] * 4 + [i32] * 4 + [vp] * 2
            lib.la_rms_norm_bwd_workspace.argtypes = [i32] * 2 + [vp]
            lib.la_rms_norm_bwd.argtypes = [vp] * 2 + [ctypes.c_float] + [vp] * 4 + [i64] * 4 + [i32] * 3 + \
                [vp, ctypes.c_size_t, vp, vp]
            lib.la_qk_norm_rope_fwd.argtypes = [vp] * 4 + [ctypes.c_float] + [vp] * 4 + [i64] * 8 + [i32] * 7 + [vp]
            lib.la_qk_norm_rope_bwd_workspace.argtypes = [i32] * 4 + [vp]
            lib.la_qk_norm_rope_bwd.argtypes = [vp] * 4 + [ctypes.c_float] + [vp] * 8 + [i64] * 12 + [i32] * 7 + \
                [vp, ctypes.c_size_t, vp]
            lib.la_attn_prefill_fwd.argtypes = [vp] * 3 + [ctypes.c_float] + [vp] * 3 + [i64] * 8 + [i32] * 6 + [vp] * 2
            lib.la_attn_prefill_bwd_workspace.argtypes = [i32] * 5 + [vp]
            lib.la_attn_prefill_bwd.argtypes = [vp] * 3 + [ctypes.c_float] + [vp] * 7 + [i64] * 16 + [i32] * 6 + \
                [vp, ctypes.c_size_t, vp, vp]
            lib.la_attn_verify_workspace.argtypes = [i32] * 5 + [vp]
            lib.la_attn_verify.argtypes = [vp] * 3 + [ctypes.c_float] + [vp] * 6 + [i64] * 15 + [i32] * 8 + \
                [vp, ctypes.c_size_t, vp, vp]
            lib.la_attn_commit.argtypes = [vp] * 9 + [i64] * 11 + [i32] * 7 + [vp] * 2
            for fn in ("la_gated_scan_workspace", "la_gated_scan_fwd", "la_gated_scan_bwd", "la_gated_decode",
                       "la_gated_verify", "la_gated_commit", "la_rms_norm_fwd", "la_rms_norm_fwd_fp8",
                       "la_rms_norm_bwd_workspace", "la_rms_norm_bwd", "la_qk_norm_rope_fwd",
                       "la_qk_norm_rope_bwd_workspace", "la_qk_norm_rope_bwd", "la_attn_prefill_fwd",
                       "la_attn_prefill_bwd_workspace", "la_attn_prefill_bwd", "la_attn_verify_workspace",
                       "la_attn_verify", "la_attn_commit"):
                getattr(lib, fn).restype = ctypes.c_int
            _lib = lib
        return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, dtype, ndim):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _prefill_args(q, k, v, slopes, h0, state_indices, cu_seqlens, o, h_final, seq_len, dev_error, stream):
    """Checks shared by the prefill entry points; returns (o, B, T, N, H, HV, D, V, pool, stream)."""
    import torch
    _check(q, "q", torch.bfloat16, 3)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    _check(slopes, "slopes", torch.float32, 1)
    _check(h0, "h0", torch.float32, 4)
    _check(h_final, "h_final", torch.float32, 4)
    _check(state_indices, "state_indices", torch.int32, 1)
    _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
    tokens, H, D = q.shape
    _, HV, V = v.shape
    if k.shape != q.shape or v.shape[0] != tokens:
        raise ValueError("q, k, v token counts / shapes disagree")
    if slopes.shape[0] != HV:
        raise ValueError("slopes must have HV entries")
    if o is None:
        o = torch.empty((tokens, HV, V), dtype=torch.bfloat16, device=q.device)
    _check(o, "o", torch.bfloat16, 3)
    if cu_seqlens is not None:
        N = cu_seqlens.shape[0] - 1
        B, T = 1, tokens
    else:
        if seq_len is None:
            raise ValueError("fixed-length mode needs seq_len")
        T = int(seq_len)
        if T == 0:
            raise ValueError("seq_len must be positive in fixed-length mode")
        if tokens % T:
            raise ValueError("tokens must be a multiple of seq_len")
        B = tokens // T
        N = B
    pool = 0
    for t in (h0, h_final):
        if t is not None:
            if tuple(t.shape[1:]) != (HV, V, D):
                raise ValueError("state tensors must be [P, HV, V, D]")
            pool = t.shape[0] if pool == 0 else min(pool, t.shape[0])
    if h0 is not None and h_final is not None and h0.shape[0] != h_final.shape[0]:
        raise ValueError("h0 and h_final must have the same number of slots")
    if state_indices is not None and state_indices.shape[0] != N:
        raise ValueError("state_indices must have N entries")
    if dev_error is not None:
        _check(dev_error, "dev_error", torch.int32, 1)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    return o, B, T, N, H, HV, D, V, pool, stream


def la_prefill_fwd(q, k, v, slopes, scale, h0=None, state_indices=None, cu_seqlens=None, o=None,
                   h_final=None, seq_len=None, schedule="auto", dev_error=None, stream=None):
    """Lightning Attention chunkwise prefill (forward) on the current CUDA device.

    q, k: bf16 [tokens, H, 128]; v: bf16 [tokens, HV, 128]; slopes: fp32 [HV];
    h0 / h_final: fp32 [P, HV, 128, 128] ([V, K] per state) or None;
    state_indices: int32 [N] or None (negative = padded sequence);
    cu_seqlens: int32 [N + 1] or None.  Without cu_seqlens the batch is fixed
    length: ``seq_len`` tokens per sequence (tokens must be a multiple of it).
    ``o`` (bf16 [tokens, HV, 128]) is allocated when not given.  h_final may be
    the same tensor as h0 (in-place state pool).  Returns ``o``.
    """
    lib = load_library()
    o, B, T, N, H, HV, D, V, pool, stream = _prefill_args(q, k, v, slopes, h0, state_indices, cu_seqlens, o,
                                                          h_final, seq_len, dev_error, stream)
    if isinstance(schedule, str):
        schedule = SCHEDULES[schedule]
    st = lib.la_prefill_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale), _ptr(h0),
                            _ptr(state_indices), _ptr(cu_seqlens), _ptr(o), _ptr(h_final),
                            int(B), int(T), int(N), int(H), int(HV), int(D), int(V), int(pool),
                            int(schedule), _ptr(dev_error), ctypes.c_void_p(stream))
    if st != 0:
        _raise(lib, st)
    return o


def la_prefill_segmented_workspace(B, T, N, HV, packed, segment_len=0):
    """(workspace bytes, resolved segment length) of la_prefill_fwd_segmented for these sizes.

    segment_len 0 = automatic (uses the current device's SM count); both values are 0 when
    the call would run la_prefill_fwd unchanged."""
    lib = load_library()
    nbytes = ctypes.c_size_t(0)
    seg = ctypes.c_int(0)
    st = lib.la_prefill_segmented_workspace(int(B), int(T), int(N), int(HV), int(bool(packed)), int(segment_len),
                                            ctypes.byref(nbytes), ctypes.byref(seg))
    if st != 0:
        _raise(lib, st)
    return nbytes.value, seg.value


def la_prefill_fwd_segmented(q, k, v, slopes, scale, h0=None, state_indices=None, cu_seqlens=None, o=None,
                             h_final=None, seq_len=None, segment_len=0, workspace=None, dev_error=None,
                             stream=None):
    """la_prefill_fwd with every sequence cut into segments of ``segment_len`` tokens (0 =
    automatic) that run in parallel from their exact initial states.

    Arguments as la_prefill_fwd; ``workspace`` is a CUDA uint8 tensor of at least
    la_prefill_segmented_workspace(...)[0] bytes, allocated here when None.  Returns ``o``."""
    import torch
    lib = load_library()
    o, B, T, N, H, HV, D, V, pool, stream = _prefill_args(q, k, v, slopes, h0, state_indices, cu_seqlens, o,
                                                          h_final, seq_len, dev_error, stream)
    if workspace is None:
        nbytes, _ = la_prefill_segmented_workspace(B, T, N, HV, cu_seqlens is not None, segment_len)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device) if nbytes else None
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, 1)
    st = lib.la_prefill_fwd_segmented(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale), _ptr(h0),
                                      _ptr(state_indices), _ptr(cu_seqlens), _ptr(o), _ptr(h_final),
                                      int(B), int(T), int(N), int(H), int(HV), int(D), int(V), int(pool),
                                      int(segment_len), _ptr(workspace),
                                      ctypes.c_size_t(0 if workspace is None else workspace.numel()),
                                      _ptr(dev_error), ctypes.c_void_p(stream))
    if st != 0:
        _raise(lib, st)
    return o


def la_prefill_fwd_segmented_static(q, k, v, slopes, scale, h0=None, state_indices=None, cu_seqlens=None,
                                    o=None, h_final=None, seq_len=None, segment_len=0, dev_error=None,
                                    stream=None):
    """la_prefill_fwd_segmented with the scratch taken from the library's built-in 16 MiB
    device buffer instead of a workspace, for callers that cannot allocate device memory.
    Calls share that buffer: calls that overlap on the GPU race.  Returns ``o``."""
    lib = load_library()
    o, B, T, N, H, HV, D, V, pool, stream = _prefill_args(q, k, v, slopes, h0, state_indices, cu_seqlens, o,
                                                          h_final, seq_len, dev_error, stream)
    st = lib.la_prefill_fwd_segmented_static(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale),
                                             _ptr(h0), _ptr(state_indices), _ptr(cu_seqlens), _ptr(o),
                                             _ptr(h_final), int(B), int(T), int(N), int(H), int(HV), int(D),
                                             int(V), int(pool), int(segment_len), _ptr(dev_error),
                                             ctypes.c_void_p(stream))
    if st != 0:
        _raise(lib, st)
    return o


def la_prefill_d256_workspace(B, T, N, HV, has_state):
    """Bytes of device workspace la_prefill_fwd_d256 needs for these sizes."""
    lib = load_library()
    nbytes = ctypes.c_size_t(0)
    st = lib.la_prefill_d256_workspace(int(B), int(T), int(N), int(HV), int(bool(has_state)), ctypes.byref(nbytes))
    if st != 0:
        _raise(lib, st)
    return nbytes.value


def la_prefill_fwd_d256(q, k, v, slopes, scale, h0=None, state_indices=None, cu_seqlens=None, o=None,
                        h_final=None, seq_len=None, workspace=None, dev_error=None, stream=None):
    """la_prefill_fwd at head dimension D = V = 256 (q, k [tokens, H, 256], v [tokens, HV, 256],
    states [P, HV, 256, 256]), run as four 128 x 128 state blocks by the D = 128 kernel.

    Arguments as la_prefill_fwd; ``workspace`` is a CUDA uint8 tensor of at least
    la_prefill_d256_workspace(...) bytes, allocated here when None.  Returns ``o``."""
    import torch
    lib = load_library()
    o, B, T, N, H, HV, D, V, pool, stream = _prefill_args(q, k, v, slopes, h0, state_indices, cu_seqlens, o,
                                                          h_final, seq_len, dev_error, stream)
    if workspace is None:
        nbytes = la_prefill_d256_workspace(B, T, N, HV, h0 is not None or h_final is not None)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    st = lib.la_prefill_fwd_d256(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale), _ptr(h0),
                                 _ptr(state_indices), _ptr(cu_seqlens), _ptr(o), _ptr(h_final), int(B), int(T),
                                 int(N), int(H), int(HV), int(D), int(V), int(pool), _ptr(workspace),
                                 ctypes.c_size_t(workspace.numel()), _ptr(dev_error), ctypes.c_void_p(stream))
    if st != 0:
        _raise(lib, st)
    return o


def la_prefill_d256_segmented_workspace(B, T, N, HV, packed, segment_len, has_state):
    """(bytes, resolved segment length) of device workspace la_prefill_fwd_d256_segmented needs."""
    lib = load_library()
    nbytes, res = ctypes.c_size_t(0), ctypes.c_int(0)
    st = lib.la_prefill_d256_segmented_workspace(int(B), int(T), int(N), int(HV), int(bool(packed)), int(segment_len),
                                                 int(bool(has_state)), ctypes.byref(nbytes), ctypes.byref(res))
    if st != 0:
        _raise(lib, st)
    return nbytes.value, res.value


def la_prefill_fwd_d256_segmented(q, k, v, slopes, scale, h0=None, state_indices=None, cu_seqlens=None, o=None,
                                  h_final=None, seq_len=None, segment_len=0, workspace=None, dev_error=None,
                                  stream=None):
    """la_prefill_fwd_d256 with every sequence cut into segments of ``segment_len`` tokens (0 =
    automatic) that run in parallel from their exact initial states; ``workspace`` as
    la_prefill_d256_segmented_workspace(...)[0] bytes, allocated here when None.  Returns ``o``."""
    import torch
    lib = load_library()
    o, B, T, N, H, HV, D, V, pool, stream = _prefill_args(q, k, v, slopes, h0, state_indices, cu_seqlens, o,
                                                          h_final, seq_len, dev_error, stream)
    if workspace is None:
        nbytes, _ = la_prefill_d256_segmented_workspace(B, T, N, HV, cu_seqlens is not None, segment_len,
                                                        h0 is not None or h_final is not None)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    st = lib.la_prefill_fwd_d256_segmented(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale), _ptr(h0),
                                           _ptr(state_indices), _ptr(cu_seqlens), _ptr(o), _ptr(h_final), int(B),
                                           int(T), int(N), int(H), int(HV), int(D), int(V), int(pool),
                                           int(segment_len), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                                           _ptr(dev_error), ctypes.c_void_p(stream))
    if st != 0:
        _raise(lib, st)
    return o


def la_prefill_bwd_workspace(B, T, H, HV, D, pool_size, has_h0, has_dh_final):
    """Bytes of device workspace la_prefill_bwd needs for these sizes."""
    lib = load_library()
    nbytes = ctypes.c_size_t(0)
    st = lib.la_prefill_bwd_workspace(int(B), int(T), int(H), int(HV), int(D), int(pool_size), int(bool(has_h0)),
                                      int(bool(has_dh_final)), ctypes.byref(nbytes))
    if st != 0:
        _raise(lib, st)
    return nbytes.value


def la_prefill_bwd(q, k, v, slopes, scale, dout, h0=None, dh_final=None, state_indices=None, cu_seqlens=None,
                   dq=None, dk=None, dv=None, dh0=None, seq_len=None, workspace=None, dev_error=None, stream=None):
    """Gradients of the prefill (include/la_backward.h): given dout = dL/do [tokens, HV, D] BF16
    and dh_final = dL/dh_final [P, HV, D, D] FP32 (or None), returns (dq, dk, dv, dh0) with the
    layouts of q, k, v and h0 (dh0 only when a tensor is passed in).  HV a multiple of H (GVA);
    the other arguments as la_prefill_fwd.  ``workspace`` is a CUDA uint8 tensor of at least
    la_prefill_bwd_workspace(...) bytes, allocated here when None."""
    import torch
    lib = load_library()
    _check(dout, "dout", torch.bfloat16, 3)
    _check(dh_final, "dh_final", torch.float32, 4)
    _check(dh0, "dh0", torch.float32, 4)
    if dout is None or dout.shape != v.shape:
        raise ValueError("dout must have the shape of v")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, name, ref in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        _check(t, name, torch.bfloat16, 3)
        if t.shape != ref.shape:
            raise ValueError(f"{name} must have the shape of its input")
    # the forward's checks and sizes: dv has the layout of o, dh0 (else dh_final) that of h_final
    _, B, T, N, H, HV, D, V, pool, stream = _prefill_args(q, k, v, slopes, h0, state_indices, cu_seqlens, dv,
                                                          dh0 if dh0 is not None else dh_final, seq_len, dev_error,
                                                          stream)
    if workspace is None:
        nbytes = la_prefill_bwd_workspace(B, T, H, HV, D, pool, h0 is not None, dh_final is not None)
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    st = lib.la_prefill_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale), _ptr(h0), _ptr(dout),
                            _ptr(dh_final), _ptr(state_indices), _ptr(cu_seqlens), _ptr(dq), _ptr(dk), _ptr(dv),
                            _ptr(dh0), int(B), int(T), int(N), int(H), int(HV), int(D), int(V), int(pool),
                            _ptr(workspace), ctypes.c_size_t(workspace.numel()), _ptr(dev_error),
                            ctypes.c_void_p(stream))
    if st != 0:
        _raise(lib, st)
    return dq, dk, dv, dh0


def _decode_common(q, k, v, slopes, state, state_indices, T, dev_error, stream):
    """Shape checks shared by the speculative-decoding ops; returns (lib, B, H, HV, pool, stream)."""
    import torch
    lib = load_library()
    for t, name, dt, nd in ((q, "q", torch.bfloat16, 3), (k, "k", torch.bfloat16, 3), (v, "v", torch.bfloat16, 3),
                            (slopes, "slopes", torch.float32, 1), (state, "state", torch.float32, 4),
                            (state_indices, "state_indices", torch.int32, 1), (dev_error, "dev_error", torch.int32, 1)):
        _check(t, name, dt, nd)
    T = int(T)
    if T < 1:
        raise ValueError("T must be >= 1")
    tokens, H, D = q.shape
    _, HV, V = v.shape
    if k.shape != q.shape or v.shape[0] != tokens or tokens % T:
        raise ValueError("q, k: [B*T, H, D]; v: [B*T, HV, V] with the same B*T")
    B = tokens // T
    if tuple(state.shape[1:]) != (HV, V, D):
        raise ValueError("state must be [P, HV, V, D]")
    if state_indices is not None and state_indices.shape[0] != B:
        raise ValueError("state_indices must have B entries")
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    return lib, B, H, HV, state.shape[0], stream


def _raise(lib, st):
    if st != 0:
        raise LaError(st, lib.la_status_string(st).decode(), lib.la_last_error().decode())


def la_decode_mtp(q, k, v, slopes, scale, state, T, state_indices=None, o=None, dev_error=None, stream=None):
    """Multi-token decode: advance each request's pooled state over its T draft tokens (in
    place) and return the outputs o (bf16 [B*T, HV, V]; D = V = 128 or 64)."""
    import torch
    lib, B, H, HV, pool, stream = _decode_common(q, k, v, slopes, state, state_indices, T, dev_error, stream)
    if o is None:
        o = torch.empty(v.shape, dtype=torch.bfloat16, device=q.device)
    _check(o, "o", torch.bfloat16, 3)
    _raise(lib, lib.la_decode_mtp(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale), _ptr(state),
                                  _ptr(state_indices), _ptr(o), B, int(T), H, HV, q.shape[2], v.shape[2], pool,
                                  _ptr(dev_error), ctypes.c_void_p(stream)))
    return o


def la_verify(q, k, v, slopes, scale, state, T, state_indices=None, o=None, kbuf=None, vbuf=None, dev_error=None,
              stream=None):
    """Parallel verify: the outputs of all T draft tokens from the pooled states, which are
    left untouched; with kbuf/vbuf (bf16 [P, T, H, D] / [P, T, HV, V]) the draft k, v
    are copied to the request's slot for la_commit.  Returns o."""
    import torch
    lib, B, H, HV, pool, stream = _decode_common(q, k, v, slopes, state, state_indices, T, dev_error, stream)
    if o is None:
        o = torch.empty(v.shape, dtype=torch.bfloat16, device=q.device)
    _check(o, "o", torch.bfloat16, 3)
    _check(kbuf, "kbuf", torch.bfloat16, 4)
    _check(vbuf, "vbuf", torch.bfloat16, 4)
    _raise(lib, lib.la_verify(_ptr(q), _ptr(k), _ptr(v), _ptr(slopes), ctypes.c_float(scale), _ptr(state),
                              _ptr(state_indices), _ptr(o), _ptr(kbuf), _ptr(vbuf), B, int(T), H, HV, q.shape[2],
                              v.shape[2], pool, _ptr(dev_error), ctypes.c_void_p(stream)))
    return o


def la_commit(state, kbuf, vbuf, accepted_len, slopes, state_indices=None, dev_error=None, stream=None):
    """Commit: advance each request's pooled state (in place) by its accepted prefix of the
    draft tokens held in kbuf/vbuf; accepted_len is int32 [B] (0 = no-op)."""
    import torch
    lib = load_library()
    _check(state, "state", torch.float32, 4)
    _check(kbuf, "kbuf", torch.bfloat16, 4)
    _check(vbuf, "vbuf", torch.bfloat16, 4)
    _check(accepted_len, "accepted_len", torch.int32, 1)
    _check(slopes, "slopes", torch.float32, 1)
    _check(state_indices, "state_indices", torch.int32, 1)
    _check(dev_error, "dev_error", torch.int32, 1)
    P, T, H, D = kbuf.shape
    HV, V = state.shape[1], state.shape[2]
    if tuple(vbuf.shape) != (P, T, HV, V) or state.shape[0] != P:
        raise ValueError("kbuf [P, T, H, D], vbuf [P, T, HV, V] and state [P, HV, V, D] must agree")
    B = accepted_len.shape[0]
    if stream is None:
        stream = torch.cuda.current_stream(state.device).cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    _raise(lib, lib.la_commit(_ptr(state), _ptr(state_indices), _ptr(kbuf), _ptr(vbuf), _ptr(accepted_len),
                              _ptr(slopes), B, T, H, HV, D, V, P, _ptr(dev_error), ctypes.c_void_p(stream)))
    return state


# ---- rows of channels: the gated recurrence (include/la_gated.h) and the RMS norm (include/la_norm.h)

# These calls serve single tokens too, where the host side is most of the time: each check is one
# expression that holds for a good argument, and the reasons are sorted out only when it fails.

def _matrix(t, name):
    """Checks of a call's leading activation matrix; returns (la_dtype, shape, rows, C, device, row stride)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype, shape = t.dtype, t.shape
    if dtype is torch.bfloat16:
        code = 0
    elif dtype is torch.float32:
        code = 1
    else:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {dtype}")
    if len(shape) != 2:
        raise ValueError(f"{name} must have 2 dims, got shape {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    rows, C = shape
    if C < 1:
        raise ValueError(f"{name} must have at least one column")
    return code, shape, rows, C, t.get_device(), _stride(t, name, rows, C)


def _stride(t, name, rows, C):
    s0, s1 = t.stride()
    if (s1 == 1 or C == 1) and s0 >= C:  # one column has no neighbour
        return s0
    if s1 != 1 and C > 1 and rows > 0:
        raise ValueError(f"the columns of {name} must be contiguous")
    if rows <= 1:
        return C
    raise ValueError(f"the row stride of {name} must be at least its {C} columns, got {s0}")


def _like(t, name, shape, dtype, dev):
    """Row stride of a matrix that must have this shape, type and device."""
    import torch
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        s0, s1 = t.stride()
        return s0 if s1 == 1 and s0 >= shape[1] else _stride(t, name, *shape)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _array(t, name, dtype, shape, dev):
    """Pointer of a contiguous tensor that must have this shape (None in it: any size), or None."""
    if t is None:
        return None
    try:
        have = t.shape
        if (t.dtype is dtype and (have == shape or (shape == (None,) and len(have) == 1)) and t.get_device() == dev
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    have = t.shape
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and len(have) == len(shape):
        if have == shape or all(w is None or h == w for h, w in zip(have, shape)):
            return t.data_ptr()
        raise ValueError(f"{name} must have shape {['any' if w is None else w for w in shape]}, got {tuple(have)}")
    _check(t, name, dtype, len(shape))
    raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _raw_stream(dev):
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without building a Stream object
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _stream_of(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, dev, stream):
    """A new tensor whose memory belongs to the stream that the call runs on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(torch.cuda.ExternalStream(_stream_of(stream, dev), device=dev)):
        return torch.empty(shape, dtype=dtype, device=dev)


def _empty_like(t, shape, dev, stream):
    """A new dense matrix of a checked matrix's shape and type (quicker by a microsecond than _empty)."""
    import torch
    return torch.empty_like(t) if stream is None else _empty(shape, t.dtype, dev, stream)


def _call(fn, dev, *args):
    """Call a C entry point with device ``dev`` current; raise on a non-OK status."""
    import torch
    if dev == torch._C._cuda_getDevice():  # a tensor on the device exists, so CUDA is up
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != 0:
        _raise(load_library(), st)


def _gated_sequences(tokens, C, dev, state_indices, cu_seqlens, seq_len, pools):
    """Batch mode of a gated scan; returns (B, T, N, pool size) and the pointers of state_indices,
    cu_seqlens and the pools."""
    import torch
    cu = None
    if cu_seqlens is not None:
        cu = _array(cu_seqlens, "cu_seqlens", torch.int32, (None,), dev)
        N = cu_seqlens.shape[0] - 1
        if N < 0:
            raise ValueError("cu_seqlens must have N + 1 entries")
        B, T = 1, tokens
    else:
        if seq_len is None:
            raise ValueError("fixed-length mode needs seq_len")
        T = int(seq_len)
        if T < 1:
            raise ValueError("seq_len must be positive in fixed-length mode")
        if tokens % T:
            raise ValueError("tokens must be a multiple of seq_len")
        B = N = tokens // T
    pool, ptrs = None, []
    for t, name in pools:
        ptrs.append(_array(t, name, torch.float32, (pool, C), dev))
        if t is not None:
            pool = t.shape[0]
    return B, T, N, pool or 0, _array(state_indices, "state_indices", torch.int32, (N,), dev), cu, ptrs


@functools.lru_cache(maxsize=1024)
def la_gated_scan_workspace(B, T, N, C, packed, dtype, backward):
    """Bytes of device workspace la_gated_scan_fwd / la_gated_scan_bwd (``backward``) needs for
    these sizes; dtype is torch.bfloat16 or torch.float32."""
    import torch
    code = {torch.bfloat16: 0, torch.float32: 1}.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    lib = load_library()
    nbytes = ctypes.c_size_t(0)
    st = lib.la_gated_scan_workspace(int(B), int(T), int(N), int(C), int(bool(packed)), code, int(bool(backward)),
                                     ctypes.byref(nbytes))
    if st != 0:
        _raise(lib, st)
    return nbytes.value


def _scan_workspace(workspace, dtype, dev, B, T, N, C, packed, backward, stream):
    """(tensor that owns it, pointer, bytes) of a scan's workspace."""
    import torch
    if workspace is None:
        nbytes = la_gated_scan_workspace(B, T, N, C, packed, dtype, backward)
        if nbytes == 0:
            return None, None, 0
        workspace = _empty(nbytes, torch.uint8, dev, stream)
        return workspace, workspace.data_ptr(), nbytes
    return workspace, _array(workspace, "workspace", torch.uint8, (None,), dev), workspace.numel()


def la_gated_scan_fwd(x, r, g, slopes, h0=None, state_indices=None, cu_seqlens=None, o=None, h_final=None,
                      seq_len=None, workspace=None, dev_error=None, stream=None):
    """Gated linear recurrence over every sequence: with u = slopes * sigmoid(r),
    h_t = exp(-u_t) h_{t-1} + sqrt(1 - exp(-2 u_t)) sigmoid(g_t) x_t and o_t = h_t.

    x, r, g: bf16 or fp32 [tokens, C], columns contiguous, any row stride (column ranges of one
    projection's output work in place); slopes: fp32 [C]; h0 / h_final: fp32 [P, C] or None
    (h_final may be h0); state_indices: int32 [N] or None (negative = padded sequence);
    cu_seqlens: int32 [N + 1] or None (then ``seq_len`` tokens per sequence).  ``o`` is allocated
    when not given; rows of padded sequences are not written.  ``workspace``: CUDA uint8, at least
    la_gated_scan_workspace(...) bytes, allocated here when None.  Returns ``o``."""
    import torch
    lib = load_library()
    code, shape, tokens, C, dev, ldx = _matrix(x, "x")
    dtype = x.dtype
    ldr, ldg = _like(r, "r", shape, dtype, dev), _like(g, "g", shape, dtype, dev)
    B, T, N, pool, idx, cu, (p0, pf) = _gated_sequences(tokens, C, dev, state_indices, cu_seqlens, seq_len,
                                                        ((h0, "h0"), (h_final, "h_final")))
    if o is None:
        o, ldo = _empty_like(x, shape, dev, stream), C
    else:
        ldo = _like(o, "o", shape, dtype, dev)
    owner, ws, nbytes = _scan_workspace(workspace, dtype, dev, B, T, N, C, cu is not None, False, stream)
    _call(lib.la_gated_scan_fwd, dev, x.data_ptr(), r.data_ptr(), g.data_ptr(),
          _array(slopes, "slopes", torch.float32, (C,), dev), p0, idx, cu, o.data_ptr(), pf, ldx, ldr, ldg, ldo, B, T, N, C,
          pool, code, ws, nbytes, _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return o


def la_gated_scan_bwd(x, r, g, slopes, o, dout, h0=None, dh_final=None, state_indices=None, cu_seqlens=None, dx=None,
                      dr=None, dg=None, dslopes=None, dh0=None, seq_len=None, workspace=None, dev_error=None,
                      stream=None):
    """Gradients of la_gated_scan_fwd: given its output ``o``, dout = dL/do and dh_final =
    dL/dh_final (fp32 [P, C] or None), returns (dx, dr, dg, dslopes, dh0); dh0 (fp32 [P, C]) only
    when a tensor is passed in.  dx, dr, dg may be column ranges of one matrix.  Rows of padded
    sequences and unselected slots are not written.  The other arguments as la_gated_scan_fwd."""
    import torch
    lib = load_library()
    code, shape, tokens, C, dev, ldx = _matrix(x, "x")
    dtype = x.dtype
    lds = [_like(t, n, shape, dtype, dev) for t, n in ((r, "r"), (g, "g"), (o, "o"), (dout, "dout"))]
    B, T, N, pool, idx, cu, (p0, pdf, pd0) = _gated_sequences(
        tokens, C, dev, state_indices, cu_seqlens, seq_len, ((h0, "h0"), (dh_final, "dh_final"), (dh0, "dh0")))
    dx, dr, dg = (_empty_like(x, shape, dev, stream) if t is None else t for t in (dx, dr, dg))
    lds += [_like(t, n, shape, dtype, dev) for t, n in ((dx, "dx"), (dr, "dr"), (dg, "dg"))]
    if dslopes is None:
        dslopes = _empty((C,), torch.float32, dev, stream)
    owner, ws, nbytes = _scan_workspace(workspace, dtype, dev, B, T, N, C, cu is not None, True, stream)
    _call(lib.la_gated_scan_bwd, dev, x.data_ptr(), r.data_ptr(), g.data_ptr(),
          _array(slopes, "slopes", torch.float32, (C,), dev), p0, o.data_ptr(), dout.data_ptr(), pdf, idx, cu,
          dx.data_ptr(), dr.data_ptr(), dg.data_ptr(), _array(dslopes, "dslopes", torch.float32, (C,), dev), pd0, ldx, *lds,
          B, T, N, C, pool, code, ws, nbytes, _array(dev_error, "dev_error", torch.int32, (None,), dev),
          _stream_of(stream, dev))
    return dx, dr, dg, dslopes, dh0


def _gated_requests(x, r, g, slopes, state, T, state_indices, dev_error):
    """Checks shared by the gated speculative-decoding ops; returns (shape, B, C, P, la_dtype, device,
    pointers of slopes, state, state_indices and dev_error, row strides)."""
    import torch
    code, shape, tokens, C, dev, ldx = _matrix(x, "x")
    dtype = x.dtype
    lds = ldx, _like(r, "r", shape, dtype, dev), _like(g, "g", shape, dtype, dev)
    if T < 1 or tokens % T:
        raise ValueError("T must be >= 1 and x must have B*T rows")
    B = tokens // T
    if state is None:
        raise TypeError("state must be a torch.Tensor")
    ptrs = (_array(slopes, "slopes", torch.float32, (C,), dev), _array(state, "state", torch.float32, (None, C), dev),
            _array(state_indices, "state_indices", torch.int32, (B,), dev),
            _array(dev_error, "dev_error", torch.int32, (None,), dev))
    return shape, B, C, state.shape[0], code, dev, ptrs, lds


def _gated_outputs(fn, x, r, g, slopes, state, T, state_indices, o, dev_error, stream):
    T = int(T)
    shape, B, C, P, code, dev, (sl, st, idx, err), lds = _gated_requests(x, r, g, slopes, state, T, state_indices,
                                                                         dev_error)
    if o is None:
        o, ldo = _empty_like(x, shape, dev, stream), C
    else:
        ldo = _like(o, "o", shape, x.dtype, dev)
    _call(fn, dev, x.data_ptr(), r.data_ptr(), g.data_ptr(), sl, st, idx, o.data_ptr(), *lds, ldo, B, T, C, P, code, err,
          _stream_of(stream, dev))
    return o


def la_gated_decode(x, r, g, slopes, state, T, state_indices=None, o=None, dev_error=None, stream=None):
    """Gated recurrence over each request's T tokens (x, r, g [B*T, C]) from its pooled state
    (fp32 [P, C]), which advances in place.  Returns the outputs o (x's type)."""
    return _gated_outputs(load_library().la_gated_decode, x, r, g, slopes, state, T, state_indices, o, dev_error,
                          stream)


def la_gated_verify(x, r, g, slopes, state, T, state_indices=None, o=None, dev_error=None, stream=None):
    """la_gated_decode's outputs (bitwise), the pooled states left untouched."""
    return _gated_outputs(load_library().la_gated_verify, x, r, g, slopes, state, T, state_indices, o, dev_error,
                          stream)


def la_gated_commit(x, r, g, slopes, state, T, accepted_len, state_indices=None, dev_error=None, stream=None):
    """Advance each request's pooled state (in place) over the first accepted_len (int32 [B]) of
    its T tokens; 0 = untouched, T = bitwise what la_gated_decode leaves.  Returns ``state``."""
    import torch
    T = int(T)
    shape, B, C, P, code, dev, (sl, st, idx, err), lds = _gated_requests(x, r, g, slopes, state, T, state_indices,
                                                                         dev_error)
    if accepted_len is None:
        raise TypeError("accepted_len must be a torch.Tensor")
    _call(load_library().la_gated_commit, dev, x.data_ptr(), r.data_ptr(), g.data_ptr(), sl, st, idx,
          _array(accepted_len, "accepted_len", torch.int32, (B,), dev), *lds, B, T, C, P, code, err,
          _stream_of(stream, dev))
    return state


def _norm_inputs(x, weight, residual, residual_out, stream):
    """Checks shared by the norm's forwards; returns (la_dtype, shape, device, pointers of residual,
    weight and residual_out, row strides of x, residual and residual_out, residual_out)."""
    import torch
    code, shape, rows, C, dev, ldx = _matrix(x, "x")
    w = _array(weight, "weight", torch.float32, (C,), dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return code, shape, dev, (None, w, None), (ldx, 0, 0), None
    ldres = _like(residual, "residual", shape, x.dtype, dev)
    if residual_out is None:
        residual_out, ldro = _empty_like(x, shape, dev, stream), C
    else:
        ldro = _like(residual_out, "residual_out", shape, x.dtype, dev)
    return code, shape, dev, (residual.data_ptr(), w, residual_out.data_ptr()), (ldx, ldres, ldro), residual_out


def la_rms_norm_fwd(x, weight, eps, residual=None, y=None, residual_out=None, dev_error=None, stream=None):
    """RMS norm of s = x + residual over the columns: y = s / sqrt(mean(s^2) + eps) * weight.

    x, residual, y, residual_out: bf16 or fp32 [rows, C] (C <= 16384), columns contiguous, any row
    stride; weight: fp32 [C].  residual_out receives s rounded to x's type and may be the residual
    itself.  Returns (y, residual_out); residual_out is None without a residual."""
    import torch
    lib = load_library()
    code, shape, dev, (res, w, ro), (ldx, ldres, ldro), residual_out = _norm_inputs(x, weight, residual, residual_out,
                                                                                    stream)
    rows, C = shape
    if y is None:
        y, ldy = _empty_like(x, shape, dev, stream), C
    else:
        ldy = _like(y, "y", shape, x.dtype, dev)
    _call(lib.la_rms_norm_fwd, dev, x.data_ptr(), res, w, eps, y.data_ptr(), ro, ldx, ldres, ldy, ldro, rows, C, code,
          _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return y, residual_out


def la_rms_norm_fwd_fp8(x, weight, eps, residual=None, group=0, y=None, scales=None, residual_out=None,
                        dev_error=None, stream=None):
    """la_rms_norm_fwd with an 8-bit output: y (torch.float8_e4m3fn [rows, C]) and FP32 scales, the
    norm's value being y * scale; one scale per row (group = 0: scales [rows, 1]) or per 128
    columns (group = 128: scales [rows, ceil(C / 128)]).  Returns (y, scales, residual_out)."""
    import torch
    lib = load_library()
    code, shape, dev, (res, w, ro), (ldx, ldres, ldro), residual_out = _norm_inputs(x, weight, residual, residual_out,
                                                                                    stream)
    rows, C = shape
    if group not in (0, 128):
        raise ValueError(f"group must be 0 or 128, got {group}")
    if y is None:
        y, ldy = _empty(shape, torch.float8_e4m3fn, dev, stream), C
    else:
        ldy = _like(y, "y", shape, torch.float8_e4m3fn, dev)
    groups = -(-C // 128) if group else 1
    if scales is None:
        scales = _empty((rows, groups), torch.float32, dev, stream)
    _call(lib.la_rms_norm_fwd_fp8, dev, x.data_ptr(), res, w, eps, y.data_ptr(),
          _array(scales, "scales", torch.float32, (rows, groups), dev), ro, ldx, ldres, ldy, ldro, rows, C, group, code,
          _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return y, scales, residual_out


@functools.lru_cache(maxsize=1024)
def la_rms_norm_bwd_workspace(rows, C):
    """Bytes of device workspace la_rms_norm_bwd needs for these sizes."""
    lib = load_library()
    nbytes = ctypes.c_size_t(0)
    st = lib.la_rms_norm_bwd_workspace(int(rows), int(C), ctypes.byref(nbytes))
    if st != 0:
        _raise(lib, st)
    return nbytes.value


def la_rms_norm_bwd(s, weight, eps, dy, dres=None, dx=None, dweight=None, workspace=None, dev_error=None,
                    stream=None):
    """Gradients of the norm of s (la_rms_norm_fwd's residual_out, or its x without a residual):
    given dy = dL/dy and dres (the gradient reaching residual_out from later layers, or None),
    returns (dx, dweight); dx is dL/dx and dL/dresidual alike, dweight fp32 [C].  ``workspace``:
    CUDA uint8, at least la_rms_norm_bwd_workspace(...) bytes, allocated here when None."""
    import torch
    lib = load_library()
    code, shape, rows, C, dev, lds = _matrix(s, "s")
    dtype = s.dtype
    lddy = _like(dy, "dy", shape, dtype, dev)
    lddres = 0 if dres is None else _like(dres, "dres", shape, dtype, dev)
    if dx is None:
        dx, lddx = _empty_like(s, shape, dev, stream), C
    else:
        lddx = _like(dx, "dx", shape, dtype, dev)
    if dweight is None:
        dweight = _empty((C,), torch.float32, dev, stream)
    if workspace is None:
        nbytes = la_rms_norm_bwd_workspace(rows, C)
        workspace = _empty(nbytes, torch.uint8, dev, stream) if nbytes else None
    else:
        nbytes = workspace.numel()
    _call(lib.la_rms_norm_bwd, dev, s.data_ptr(), _array(weight, "weight", torch.float32, (C,), dev), eps, dy.data_ptr(),
          None if dres is None else dres.data_ptr(), dx.data_ptr(),
          _array(dweight, "dweight", torch.float32, (C,), dev), lds, lddy, lddres, lddx, rows, C, code,
          _array(workspace, "workspace", torch.uint8, (None,), dev), nbytes,
          _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return dx, dweight


# ---- queries, keys and values as heads: norm and rotation (include/la_rotary.h), softmax attention
#      (include/la_attention.h)

# As above, a check is one expression that holds for a good argument.

def _heads(t, name, dtype=None, dev=None, shape=None):
    """Checks of a tensor [tokens, heads, D] with contiguous D (dtype, dev, shape None: any); returns
    (pointer, token stride, head stride)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            ld, hs, one = t.stride()
            if one == 1:
                return t.data_ptr(), ld, hs
    except AttributeError:
        pass
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    have = t.shape
    if len(have) != 3:
        raise ValueError(f"{name} must have 3 dims, got shape {tuple(have)}")
    if shape is not None and have != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(have)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    ld, hs, one = t.stride()
    if one != 1 and have[2] > 1 and have[0] * have[1] > 0:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return t.data_ptr(), ld, hs


def _out_heads(t, like, name, dtype, dev, stream):
    """(tensor, pointer, strides) of an output of a checked tensor's shape and type, a new dense tensor
    when not given."""
    shape = like.shape
    if t is not None:
        return t, *_heads(t, name, dtype, dev, shape)
    if stream is None:
        import torch
        t = torch.empty_like(like)  # the quickest of torch's ways; dense, in the order of like's strides
        ld, hs, _ = t.stride()
        return t, t.data_ptr(), ld, hs
    t = _empty(shape, dtype, dev, stream)
    return t, t.data_ptr(), shape[1] * shape[2], shape[2]


def _out_array(t, name, shape, dev, stream):
    """(tensor, pointer) of a contiguous fp32 output, a new tensor when not given."""
    import torch
    if t is not None:
        return t, _array(t, name, torch.float32, shape, dev)
    t = _empty(shape, torch.float32, dev, stream)
    return t, t.data_ptr()


def _count(t):
    """Heads of a tensor that is about to be checked."""
    try:
        return t.shape[1]
    except (AttributeError, IndexError):
        return None


def _qk(q, k):
    """Checks shared by the norm and rotation calls; returns (la_dtype, dtype, device, q shape, k shape, q, k)."""
    import torch
    qs = _heads(q, "q")
    dtype, dev = q.dtype, q.get_device()
    code = 0 if dtype is torch.bfloat16 else 1 if dtype is torch.float32 else None
    if code is None:
        raise TypeError(f"q must be torch.bfloat16 or torch.float32, got {dtype}")
    tokens, H, D = q.shape
    ks = _heads(k, "k", dtype, dev, (tokens, _count(k), D))
    return code, dtype, dev, q.shape, k.shape, qs, ks


def _rotation(positions, inv_freq, tokens, dev):
    """(pointer of positions, pointer of inv_freq, R)."""
    import torch
    if inv_freq is None:
        if positions is not None:
            raise ValueError("positions needs inv_freq")
        return None, None, 0
    if positions is None:
        raise ValueError("inv_freq needs positions")
    return (_array(positions, "positions", torch.int32, (tokens,), dev),
            _array(inv_freq, "inv_freq", torch.float32, (None,), dev), 2 * inv_freq.shape[0])


def la_qk_norm_rope_fwd(q, k, q_weight, k_weight, eps, positions=None, inv_freq=None, interleaved=False, q_out=None,
                        k_out=None, stream=None):
    """RMS norm of every query and key head over its D elements, then the position rotation of the
    first R of them: pair i by the angle positions[t] * inv_freq[i] (pairs (i, i + R/2), or (2i, 2i + 1)
    with ``interleaved``).

    q: bf16 or fp32 [tokens, H, D]; k: [tokens, HK, D] (D = 64, 128, 256), D contiguous, any strides
    between tokens and heads (column ranges of one projection's output work in place); q_weight,
    k_weight: fp32 [D] or None (ones); positions: int32 [tokens]; inv_freq: fp32 [R / 2] (both None: no
    rotation).  q_out and k_out may be q and k themselves.  Returns (q_out, k_out)."""
    import torch
    lib = _lib or load_library()
    code, dtype, dev, (tokens, H, D), (_, HK, _), (pq, ldq, hsq), (pk, ldk, hsk) = _qk(q, k)
    pos, freq, R = _rotation(positions, inv_freq, tokens, dev)
    q_out, pqo, ldqo, hsqo = _out_heads(q_out, q, "q_out", dtype, dev, stream)
    k_out, pko, ldko, hsko = _out_heads(k_out, k, "k_out", dtype, dev, stream)
    _call(lib.la_qk_norm_rope_fwd, dev, pq, pk, _array(q_weight, "q_weight", torch.float32, (D,), dev),
          _array(k_weight, "k_weight", torch.float32, (D,), dev), eps, pos, freq, pqo, pko, ldq, hsq, ldk, hsk, ldqo, hsqo,
          ldko, hsko, tokens, H, HK, D, R, int(bool(interleaved)), code, _stream_of(stream, dev))
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def la_qk_norm_rope_bwd_workspace(tokens, H, HK, D):
    """Bytes of device workspace la_qk_norm_rope_bwd needs for these sizes."""
    return _bytes_of(load_library().la_qk_norm_rope_bwd_workspace, tokens, H, HK, D)


def _bytes_of(fn, *sizes):
    nbytes = ctypes.c_size_t(0)
    st = fn(*(int(n) for n in sizes), ctypes.byref(nbytes))
    if st != 0:
        _raise(load_library(), st)
    return nbytes.value


class _Scratch:
    """Memory of torch's allocator for one call on a stream, free for later work on it once the call has
    returned; without a tensor around it, which took four of the microseconds of a call (with: 4.4, without: 0.8)."""
    __slots__ = ("ptr", "delete")

    def __init__(self, ptr, delete):
        self.ptr, self.delete = ptr, delete

    def __del__(self):
        self.delete(self.ptr)


def _workspace(workspace, query, sizes, dev, stream):
    """(what owns it, pointer, bytes) of a call's workspace."""
    import torch
    if workspace is not None:
        return workspace, _array(workspace, "workspace", torch.uint8, (None,), dev), workspace.numel()
    nbytes = query(*sizes)
    C = torch._C
    alloc = getattr(C, "_cuda_cudaCachingAllocator_raw_alloc", None)
    delete = getattr(C, "_cuda_cudaCachingAllocator_raw_delete", None)
    if alloc is not None and delete is not None and nbytes > 0 and dev == C._cuda_getDevice():
        scratch = _Scratch(alloc(nbytes, _stream_of(stream, dev)), delete)
        return scratch, scratch.ptr, nbytes
    workspace = _empty(nbytes, torch.uint8, dev, stream)
    return workspace, workspace.data_ptr(), nbytes


def la_qk_norm_rope_bwd(q, k, q_weight, k_weight, eps, dq_out, dk_out, positions=None, inv_freq=None, interleaved=False,
                        dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None, stream=None):
    """Gradients of la_qk_norm_rope_fwd for its inputs q and k, given those of its outputs; returns
    (dq, dk, dq_weight, dk_weight).  dq and dk may be dq_out and dk_out themselves.  ``workspace``:
    CUDA uint8, at least la_qk_norm_rope_bwd_workspace(...) bytes, allocated here when None."""
    import torch
    lib = _lib or load_library()
    code, dtype, dev, (tokens, H, D), (_, HK, _), (pq, ldq, hsq), (pk, ldk, hsk) = _qk(q, k)
    pos, freq, R = _rotation(positions, inv_freq, tokens, dev)
    pgq, ldgq, hsgq = _heads(dq_out, "dq_out", dtype, dev, q.shape)
    pgk, ldgk, hsgk = _heads(dk_out, "dk_out", dtype, dev, k.shape)
    dq, pdq, lddq, hsdq = _out_heads(dq, q, "dq", dtype, dev, stream)
    dk, pdk, lddk, hsdk = _out_heads(dk, k, "dk", dtype, dev, stream)
    dq_weight, pdwq = _out_array(dq_weight, "dq_weight", (D,), dev, stream)
    dk_weight, pdwk = _out_array(dk_weight, "dk_weight", (D,), dev, stream)
    owner, ws, nbytes = _workspace(workspace, la_qk_norm_rope_bwd_workspace, (tokens, H, HK, D), dev, stream)
    _call(lib.la_qk_norm_rope_bwd, dev, pq, pk, _array(q_weight, "q_weight", torch.float32, (D,), dev),
          _array(k_weight, "k_weight", torch.float32, (D,), dev), eps, pos, freq, pgq, pgk, pdq, pdk, pdwq,
          pdwk, ldq, hsq, ldk, hsk, ldgq, hsgq, ldgk, hsgk, lddq, hsdq, lddk, hsdk, tokens, H, HK, D, R,
          int(bool(interleaved)), code, ws, nbytes, _stream_of(stream, dev))
    return dq, dk, dq_weight, dk_weight


def _qkv(q, k, v):
    """Checks shared by the attention calls; returns (device, q and k shapes, q, k, v as _heads)."""
    import torch
    qs = _heads(q, "q", torch.bfloat16)
    dev = q.get_device()
    shape = q.shape
    kshape = (shape[0], _count(k), shape[2])
    ks = _heads(k, "k", torch.bfloat16, dev, kshape)
    return dev, shape, kshape, qs, ks, _heads(v, "v", torch.bfloat16, dev, kshape)


def _prompt_sequences(tokens, dev, cu_seqlens, seq_len):
    """(B, T, N, pointer of cu_seqlens) of a prompt call."""
    import torch
    if cu_seqlens is not None:
        N = cu_seqlens.shape[0] - 1 if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dim() == 1 else 0
        cu = _array(cu_seqlens, "cu_seqlens", torch.int32, (None,), dev)
        if N < 0:
            raise ValueError("cu_seqlens must have N + 1 entries")
        return 1, tokens, N, cu
    if seq_len is None:
        raise ValueError("fixed-length mode needs seq_len")
    T = int(seq_len)
    if T < 1:
        raise ValueError("seq_len must be positive in fixed-length mode")
    if tokens % T:
        raise ValueError("tokens must be a multiple of seq_len")
    return tokens // T, T, tokens // T, None


def la_attn_prefill_fwd(q, k, v, scale, cu_seqlens=None, seq_len=None, o=None, lse=None, dev_error=None, stream=None):
    """Causal softmax attention over whole sequences with grouped heads.

    q: bf16 [tokens, H, D]; k, v: bf16 [tokens, HK, D] (D = 64, 128; H a multiple of HK), D contiguous,
    strides between tokens and heads multiples of 8 elements, 16-byte aligned; cu_seqlens: int32
    [N + 1] or None (then ``seq_len`` tokens per sequence).  Rows of no sequence are not written.
    Returns (o, lse), lse fp32 [H, tokens], both allocated when not given."""
    import torch
    lib = _lib or load_library()
    dev, (tokens, H, D), (_, HK, _), (pq, ldq, hsq), (pk, ldk, hsk), (pv, ldv, hsv) = _qkv(q, k, v)
    B, T, N, cu = _prompt_sequences(tokens, dev, cu_seqlens, seq_len)
    o, po, ldo, hso = _out_heads(o, q, "o", torch.bfloat16, dev, stream)
    lse, plse = _out_array(lse, "lse", (H, tokens), dev, stream)
    _call(lib.la_attn_prefill_fwd, dev, pq, pk, pv, scale, cu, po, plse, ldq, hsq, ldk, hsk, ldv, hsv,
          ldo, hso, B, T, N, H, HK, D, _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return o, lse


@functools.lru_cache(maxsize=1024)
def la_attn_prefill_bwd_workspace(B, T, H, HK, D):
    """Bytes of device workspace la_attn_prefill_bwd needs for B sequences of T tokens (packed: 1, tokens)."""
    return _bytes_of(load_library().la_attn_prefill_bwd_workspace, B, T, H, HK, D)


def la_attn_prefill_bwd(q, k, v, scale, o, lse, dout, cu_seqlens=None, seq_len=None, dq=None, dk=None, dv=None,
                        workspace=None, dev_error=None, stream=None):
    """Gradients of la_attn_prefill_fwd, given its outputs o and lse and dout = dL/do; returns
    (dq, dk, dv).  Rows of no sequence are not written.  ``workspace``: CUDA uint8, at least
    la_attn_prefill_bwd_workspace(...) bytes, allocated here when None."""
    import torch
    lib = _lib or load_library()
    bf16 = torch.bfloat16
    dev, (tokens, H, D), (_, HK, _), (pq, ldq, hsq), (pk, ldk, hsk), (pv, ldv, hsv) = _qkv(q, k, v)
    B, T, N, cu = _prompt_sequences(tokens, dev, cu_seqlens, seq_len)
    po, ldo, hso = _heads(o, "o", bf16, dev, q.shape)
    pg, ldg, hsg = _heads(dout, "dout", bf16, dev, q.shape)
    if lse is None:
        raise TypeError("lse must be a torch.Tensor")
    plse = _array(lse, "lse", torch.float32, (H, tokens), dev)
    dq, pdq, lddq, hsdq = _out_heads(dq, q, "dq", bf16, dev, stream)
    dk, pdk, lddk, hsdk = _out_heads(dk, k, "dk", bf16, dev, stream)
    dv, pdv, lddv, hsdv = _out_heads(dv, v, "dv", bf16, dev, stream)
    owner, ws, nbytes = _workspace(workspace, la_attn_prefill_bwd_workspace, (B, T, H, HK, D), dev, stream)
    _call(lib.la_attn_prefill_bwd, dev, pq, pk, pv, scale, po, plse, pg, cu, pdq, pdk, pdv, ldq, hsq, ldk, hsk, ldv, hsv,
          ldo, hso, ldg, hsg, lddq, hsdq, lddk, hsdk, lddv, hsdv, B, T, N, H, HK, D, ws, nbytes,
          _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return dq, dk, dv


def _pages(t, name, HK, D, dev):
    """(strides between pages, tokens and heads, shape) of a checked half of a cache."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    have = t.shape
    if len(have) != 4 or have[2] != HK or have[3] != D:
        raise ValueError(f"{name} must have shape [pages, page_size, {HK}, {D}], got {tuple(have)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    pages, tokens, heads, one = t.stride()
    if one != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return pages, tokens, heads, have


def _cache(k_cache, v_cache, HK, D, cache_lens, page_table, B, dev):
    """Checks of a key/value cache; returns (pointers of k_cache, v_cache, cache_lens, page_table; the
    strides; (pages, page_size, table_width))."""
    import torch
    kp, kt, kh, shape = _pages(k_cache, "k_cache", HK, D, dev)
    vp, vt, vh, vshape = _pages(v_cache, "v_cache", HK, D, dev)
    if vshape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if cache_lens is None:
        raise TypeError("cache_lens must be a torch.Tensor")
    lens = _array(cache_lens, "cache_lens", torch.int32, (B,), dev)
    pages, size, _, _ = shape
    table, width, ld = None, 0, 0
    if page_table is not None:
        if not isinstance(page_table, torch.Tensor):
            raise TypeError("page_table must be a torch.Tensor")
        if page_table.dtype is not torch.int32:
            raise TypeError(f"page_table must be torch.int32, got {page_table.dtype}")
        if page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError(f"page_table must have shape [{B}, width], got {tuple(page_table.shape)}")
        if page_table.get_device() != dev:
            raise ValueError(f"page_table must be on cuda:{dev}, got {page_table.device}")
        width, (ld, one) = page_table.shape[1], page_table.stride()
        if width < 1:  # (its pointer is null, which would mean no table)
            raise ValueError("page_table must have at least one column")
        if one != 1 and width > 1:
            raise ValueError("the rows of page_table must be contiguous")
        table = page_table.data_ptr()
    return (k_cache.data_ptr(), v_cache.data_ptr(), lens, table), (kp, kt, kh, vp, vt, vh, ld), (pages, size, width)


@functools.lru_cache(maxsize=1024)
def la_attn_verify_workspace(B, T, H, HK, D):
    """Bytes of device workspace la_attn_verify needs for these sizes."""
    return _bytes_of(load_library().la_attn_verify_workspace, B, T, H, HK, D)


def la_attn_verify(q, k, v, scale, k_cache, v_cache, cache_lens, T, page_table=None, mask=None, o=None, workspace=None,
                   dev_error=None, stream=None):
    """Softmax attention of each request's T drafted tokens over its cache and the drafted tokens
    themselves, the cache left untouched (T = 1: decode).

    q: bf16 [B*T, H, D]; k, v: bf16 [B*T, HK, D]; k_cache, v_cache: bf16 [pages, page_size, HK, D], any
    strides between pages, tokens and heads that are multiples of 8; cache_lens: int32 [B] (negative =
    padded request, nothing written); page_table: int32 [B, width] or None (request b has page b);
    mask: int64 [B, T] or None: bit u of mask[b, t] lets token t see drafted token u (None: tokens
    0 .. t).  ``workspace``: CUDA uint8, at least la_attn_verify_workspace(...) bytes, allocated here
    when None.  Returns ``o``."""
    import torch
    lib = _lib or load_library()
    T = int(T)
    dev, (tokens, H, D), (_, HK, _), (pq, ldq, hsq), (pk, ldk, hsk), (pv, ldv, hsv) = _qkv(q, k, v)
    if T < 1 or tokens % T:
        raise ValueError("T must be >= 1 and q must have B*T rows")
    B = tokens // T
    (pkc, pvc, lens, table), strides, sizes = _cache(k_cache, v_cache, HK, D, cache_lens, page_table, B, dev)
    o, po, ldo, hso = _out_heads(o, q, "o", torch.bfloat16, dev, stream)
    owner, ws, nbytes = _workspace(workspace, la_attn_verify_workspace, (B, T, H, HK, D), dev, stream)
    _call(lib.la_attn_verify, dev, pq, pk, pv, scale, pkc, pvc, lens, table, _array(mask, "mask", torch.int64, (B, T), dev),
          po, ldq, hsq, ldk, hsk, ldv, hsv, ldo, hso, *strides, B, T, H, HK, D, *sizes, ws, nbytes,
          _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return o


def la_attn_commit(k, v, k_cache, v_cache, cache_lens, T=None, cu_seqlens=None, accepted_len=None, path=None,
                   page_table=None, dev_error=None, stream=None):
    """Write tokens' keys and values (bf16 [tokens, HK, D]) into the cache behind each request's
    cache_lens tokens (the caller then advances cache_lens).

    With ``T``: request b has tokens b*T .. and commits accepted_len[b] of them (int32 [B]; None: all),
    those that path[b] lists (int32 [B, T]; None: the first).  With ``cu_seqlens`` (int32 [B + 1]):
    request b commits tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1, as after a prompt.  The cache as
    in la_attn_verify.  Returns (k_cache, v_cache)."""
    import torch
    lib = _lib or load_library()
    pk, ldk, hsk = _heads(k, "k", torch.bfloat16)
    dev = k.get_device()
    tokens, HK, D = k.shape
    pv, ldv, hsv = _heads(v, "v", torch.bfloat16, dev, k.shape)
    if (T is None) == (cu_seqlens is None):
        raise ValueError("give either T or cu_seqlens")
    if cu_seqlens is not None:
        cu = _array(cu_seqlens, "cu_seqlens", torch.int32, (None,), dev)
        B, T = cu_seqlens.shape[0] - 1, tokens
        if B < 0:
            raise ValueError("cu_seqlens must have B + 1 entries")
        if accepted_len is not None or path is not None:
            raise ValueError("accepted_len and path go with T, not with cu_seqlens")
    else:
        cu, T = None, int(T)
        if T < 1 or tokens % T:
            raise ValueError("T must be >= 1 and k must have B*T rows")
        B = tokens // T
    (pkc, pvc, lens, table), strides, sizes = _cache(k_cache, v_cache, HK, D, cache_lens, page_table, B, dev)
    _call(lib.la_attn_commit, dev, pk, pv, pkc, pvc, lens, cu, _array(accepted_len, "accepted_len", torch.int32, (B,), dev),
          _array(path, "path", torch.int32, (B, T), dev), table, ldk, hsk, ldv, hsv, *strides, B, T, HK, D, *sizes,
          _array(dev_error, "dev_error", torch.int32, (None,), dev), _stream_of(stream, dev))
    return k_cache, v_cache


def la_prefill_fwd_raw(*args):
    """Call the C entry point with raw integers / pointers (argument order of the header)."""
    return load_library().la_prefill_fwd(*args)
