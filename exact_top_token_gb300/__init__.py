"""exact_top_token_gb300 -- exact top-k indexer selection without a score
table (HyTopK), selection replay and the two-pass comparison path, for one
NVIDIA GB300 (sm_103a).

This module is a thin ctypes binding over the C ABI declared in
``include/hytopk.h`` (``_build/libhytopk.so``): it checks dtypes, allocates
outputs and workspace with torch on the tensors' device and passes raw
pointers and the current CUDA stream. Every step of the computation runs in
the library's kernels; there is no CPU path. If the compiled library is
missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

__all__ = ["build", "load", "select", "select_twopass", "replay", "select_workspace_size",
           "select_fallback_chunks",
           "select_sharded", "select_varlen", "replay_varlen", "replay_backward",
           "replay_backward_varlen",
           "rope", "rope_frequencies", "cache_write", "cache_read", "attend", "attend_backward",
           "twopass_workspace_size", "sample_plan", "HytopkError", "STATUS", "PHASES", "Stats",
           "symbols"]

MAX_RECOVERY_ROWS = 64
PHASES = ("prep", "threshold", "filter", "check", "select", "recover")
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape or dtype",
          3: "workspace too small", 4: "CUDA error", 5: "device pointer misaligned"}
DEV_REPLAY_BAD_INDEX = 0x1
DEV_BAD_SCALE = 0x2
DEV_BAD_POSITION = 0x4
DEV_BAD_INDEX = DEV_REPLAY_BAD_INDEX
DEV_NONFINITE = 0x8
DEV_WAIT_TIMEOUT = 0x80000000  # a bounded wait gave up: the call's outputs are undefined
BF16, E4M3, E4M3_BF16 = 0, 1, 2  # E4M3_BF16: e4m3 q (with q_scale), bf16 k

ELEM_BF16, ELEM_E4M3, ELEM_F32 = 0, 1, 2

# the C-ABI symbols declared in include/hytopk.h
symbols = ("hytopk_select_workspace_size", "hytopk_select_fallback_chunks", "hytopk_select",
           "hytopk_select_ex", "hytopk_replay",
           "hytopk_twopass_workspace_size", "hytopk_select_twopass", "hytopk_select_noalloc",
           "hytopk_select_sharded_workspace_size", "hytopk_select_sharded",
           "hytopk_replay_backward", "hytopk_select_varlen_workspace_size",
           "hytopk_select_varlen", "hytopk_replay_varlen", "hytopk_replay_grouped",
           "hytopk_replay_backward_varlen", "hytopk_sample_plan",
           "hytopk_rope", "hytopk_cache_write", "hytopk_cache_read", "hytopk_attend",
           "hytopk_attend_backward",
           "hytopk_status_string", "hytopk_version")


class HytopkError(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class Stats(ctypes.Structure):
    _fields_ = [("n_failed", ctypes.c_int32), ("n_overflow", ctypes.c_int32),
                ("n_under_k", ctypes.c_int32), ("fallback_used", ctypes.c_int32),
                ("total_candidates", ctypes.c_int64), ("device_status", ctypes.c_uint32),
                ("n_queries", ctypes.c_int32)]


class SelectOptions(ctypes.Structure):
    _fields_ = [("threshold_override", ctypes.c_void_p), ("phase_events", ctypes.c_void_p),
                ("reverse_schedule", ctypes.c_int), ("reserved", ctypes.c_int)]


class RopeParams(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("rot", ctypes.c_int), ("first", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("inverse", ctypes.c_int), ("mscale", ctypes.c_float)]


_lib = None


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA library for sm_103a (in-tree)."""
    return _build.build(force=force, verbose=verbose)


def load(path: str | None = None):
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"the HyTopK CUDA library is not built ({path}); "
                           "call exact_top_token_gb300.build() first")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.hytopk_select_workspace_size.restype = Z
    lib.hytopk_select_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.hytopk_select_fallback_chunks.restype = ctypes.c_int32
    lib.hytopk_select_fallback_chunks.argtypes = [I, I, I, I, I, I, I]
    sel = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, I, P, Z, P]
    lib.hytopk_select.restype = I
    lib.hytopk_select.argtypes = sel + [P]
    lib.hytopk_select_ex.restype = I
    lib.hytopk_select_ex.argtypes = sel + [P, P]
    lib.hytopk_replay.restype = I
    lib.hytopk_replay.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, P]
    lib.hytopk_replay_grouped.restype = I
    lib.hytopk_replay_grouped.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P]
    lib.hytopk_twopass_workspace_size.restype = Z
    lib.hytopk_twopass_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.hytopk_select_twopass.restype = I
    lib.hytopk_select_twopass.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, Z, P, P]
    lib.hytopk_select_sharded_workspace_size.restype = Z
    lib.hytopk_select_sharded_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
    lib.hytopk_select_sharded.restype = I
    lib.hytopk_select_sharded.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, I, P, Z, P,
                                          P]
    lib.hytopk_replay_backward.restype = I
    lib.hytopk_replay_backward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, P, P]
    lib.hytopk_select_varlen_workspace_size.restype = Z
    lib.hytopk_select_varlen_workspace_size.argtypes = [P, P, I, I, I, I, I, I]
    lib.hytopk_select_varlen.restype = I
    lib.hytopk_select_varlen.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, I, P, Z, P,
                                         P]
    lib.hytopk_replay_varlen.restype = I
    lib.hytopk_replay_varlen.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, P]
    lib.hytopk_replay_backward_varlen.restype = I
    lib.hytopk_replay_backward_varlen.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, P, P,
                                                  P, P]
    S, F = ctypes.c_int64, ctypes.c_float
    lib.hytopk_rope.restype = I
    lib.hytopk_rope.argtypes = [P, S, S, I, I, I, I, P, P, S, S, P, P]
    lib.hytopk_cache_write.restype = I
    lib.hytopk_cache_write.argtypes = [P, S, S, I, I, I, I, P, P, P, I, P, I, P, P]
    lib.hytopk_cache_read.restype = I
    lib.hytopk_cache_read.argtypes = [P, I, P, I, P, I, I, I, P, I, P, P]
    lib.hytopk_attend.restype = I
    lib.hytopk_attend.argtypes = [P, S, P, S, P, P, S, P, P, I, I, I, I, I, I, I, F, P, I, P, P, P]
    lib.hytopk_attend_backward.restype = I
    lib.hytopk_attend_backward.argtypes = [P, S, P, S, P, S, P, P, I, P, P, I, I, I, I, I, I, F, P,
                                           P, P, I, P, P]
    lib.hytopk_sample_plan.restype = ctypes.c_int32
    lib.hytopk_sample_plan.argtypes = [ctypes.c_int64, ctypes.c_int32, P, P]
    lib.hytopk_status_string.restype = ctypes.c_char_p
    lib.hytopk_status_string.argtypes = [I]
    lib.hytopk_version.restype = I
    lib.hytopk_version.argtypes = []
    if path == _build.LIB:
        _lib = lib
    return lib


# ---- argument marshalling -----------------------------------------------------------

def _dtype_code(q, k):
    import torch

    kinds = {torch.bfloat16: BF16, torch.int16: BF16, torch.uint16: BF16,
             torch.float8_e4m3fn: E4M3, torch.uint8: E4M3}
    if q.dtype not in kinds or k.dtype not in kinds:
        raise TypeError("q and k must be bfloat16 (or its 16-bit patterns) or float8_e4m3fn "
                        "(or its 8-bit codes)")
    dq, dk = kinds[q.dtype], kinds[k.dtype]
    if dq == dk:
        return dq
    if dq == E4M3 and dk == BF16:
        return E4M3_BF16
    raise TypeError("bf16 q with e4m3 k is not supported (e4m3 q with bf16 k is)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    import torch

    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check_tensor(name, t, device, dtype=None, shape=None):
    if t is None:
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _common(q, q_scale, k, k_scale, w):
    import torch

    dt = _dtype_code(q, k)
    n, H, d = q.shape
    L = k.shape[0]
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check_tensor("q", q, dev)
    _check_tensor("k", k, dev, shape=(L, d))
    _check_tensor("w", w, dev, torch.float32, (n, H))
    _check_tensor("q_scale", q_scale, dev, torch.float32, (n, H))
    _check_tensor("k_scale", k_scale, dev, torch.float32, (L,))
    return dt, n, L, H, d, dev


def sample_plan(ctx: int, k_top: int):
    """(positions, r): the sample positions of a query with ctx visible keys
    and the rank of its threshold among them (host computation in the library)."""
    import numpy as np

    lib = load()
    out = np.zeros(8192, dtype=np.int32)
    r = ctypes.c_int32(0)
    m = lib.hytopk_sample_plan(int(ctx), int(k_top), out.ctypes.data_as(ctypes.c_void_p),
                               ctypes.byref(r))
    return out[:m].copy(), int(r.value)


def select_workspace_size(n, L, H, d, k_top, capacity=0, dtype=BF16) -> int:
    return int(load().hytopk_select_workspace_size(n, L, H, d, k_top, capacity, dtype))


def select_fallback_chunks(n, L, H, d, k_top, capacity=0, dtype=BF16) -> int:
    """Score-table chunks (table writer + read-back launch pairs) of
    hytopk_select's fallback; -1 for invalid arguments."""
    return int(load().hytopk_select_fallback_chunks(n, L, H, d, k_top, capacity, dtype))


def twopass_workspace_size(n, L, H, d, k_top, dtype=BF16, rows_per_chunk=0) -> int:
    return int(load().hytopk_twopass_workspace_size(n, L, H, d, k_top, dtype, rows_per_chunk))


def _workspace(nbytes, device, workspace):
    import torch

    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise HytopkError(3, "workspace")
        return workspace
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    if ws.data_ptr() % 256:
        raise RuntimeError("allocator returned a workspace that is not 256-byte aligned")
    return ws


def select(q, k, w, positions, k_top, *, q_scale=None, k_scale=None, capacity=0,
           scores=True, stats=False, workspace=None, threshold_override=None,
           phase_events=None, reverse_schedule=False, out=None, stream=None):
    """Exact top-k key positions per query (HyTopK).

    Returns ``(idx [n,k] int32, scores [n,k] f32 or None, stats or None)``.
    ``stats`` (when requested) is a device int32 tensor holding the
    ``hytopk_stats`` struct; read it with :func:`read_stats`.
    """
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    _check_tensor("positions", positions, dev, torch.int32, (n,))
    if out is not None:
        idx, sc = out
    else:
        idx = torch.empty((n, k_top), dtype=torch.int32, device=dev)
        sc = torch.empty((n, k_top), dtype=torch.float32, device=dev) if scores else None
    need = lib.hytopk_select_workspace_size(n, L, H, d, k_top, capacity, dt)
    if need == 0:
        raise HytopkError(2, "hytopk_select_workspace_size")
    ws = _workspace(need, dev, workspace)
    st = torch.zeros(8, dtype=torch.int32, device=dev) if stats else None
    opts = None
    ev_array = None
    if threshold_override is not None or phase_events is not None or reverse_schedule:
        opts = SelectOptions()
        if threshold_override is not None:
            _check_tensor("threshold_override", threshold_override, dev, torch.float32, (n,))
            opts.threshold_override = threshold_override.data_ptr()
        if phase_events is not None:
            if len(phase_events) != len(PHASES) + 1:
                raise ValueError(f"phase_events needs {len(PHASES) + 1} events")
            ev_array = (ctypes.c_void_p * len(phase_events))(
                *[e.cuda_event for e in phase_events])
            opts.phase_events = ctypes.cast(ev_array, ctypes.c_void_p).value
        opts.reverse_schedule = int(bool(reverse_schedule))
    status = lib.hytopk_select_ex(
        _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(positions), n, L, H, d,
        k_top, dt, _ptr(idx), _ptr(sc), capacity, _ptr(ws), ws.numel(), _ptr(st),
        ctypes.byref(opts) if opts is not None else None, _stream(dev, stream))
    if status != 0:
        raise HytopkError(status, "hytopk_select")
    return idx, sc, st


def select_sharded_workspace_size(n, L, H, d, k_top, num_shards, capacity=0, dtype=BF16) -> int:
    return int(load().hytopk_select_sharded_workspace_size(n, L, H, d, k_top, capacity, dtype,
                                                           num_shards))


def select_sharded(q, k, w, positions, k_top, num_shards, *, q_scale=None, k_scale=None,
                   capacity=0, scores=True, stats=False, workspace=None, stream=None):
    """Key-sharded exact selection: one HyTopK selection per key range, then a
    merge per query. Same outputs as :func:`select`."""
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    _check_tensor("positions", positions, dev, torch.int32, (n,))
    idx = torch.empty((n, k_top), dtype=torch.int32, device=dev)
    sc = torch.empty((n, k_top), dtype=torch.float32, device=dev) if scores else None
    need = lib.hytopk_select_sharded_workspace_size(n, L, H, d, k_top, capacity, dt, num_shards)
    if need == 0:
        raise HytopkError(2, "hytopk_select_sharded_workspace_size")
    ws = _workspace(need, dev, workspace)
    st = torch.zeros(8, dtype=torch.int32, device=dev) if stats else None
    status = lib.hytopk_select_sharded(
        _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(positions), n, L, H, d,
        k_top, dt, num_shards, _ptr(idx), _ptr(sc), capacity, _ptr(ws), ws.numel(), _ptr(st),
        _stream(dev, stream))
    if status != 0:
        raise HytopkError(status, "hytopk_select_sharded")
    return idx, sc, st


def _offsets(cu, name):
    """Host int32 copy of a B+1 offset array (list, numpy or tensor)."""
    import numpy as np

    if hasattr(cu, "cpu"):
        cu = cu.cpu().numpy()
    a = np.ascontiguousarray(np.asarray(cu, dtype=np.int32))
    if a.ndim != 1 or a.size < 2:
        raise ValueError(f"{name} must hold B+1 offsets")
    return a


def _cu_ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def select_varlen_workspace_size(cu_q, cu_k, H, d, k_top, capacity=0, dtype=BF16) -> int:
    cq, ck = _offsets(cu_q, "cu_q"), _offsets(cu_k, "cu_k")
    if cq.size != ck.size:
        raise ValueError("cu_q and cu_k must have the same length")
    return int(load().hytopk_select_varlen_workspace_size(_cu_ptr(cq), _cu_ptr(ck), cq.size - 1, H,
                                                          d, k_top, capacity, dtype))


def select_varlen(q, k, w, positions, cu_q, cu_k, k_top, *, q_scale=None, k_scale=None,
                  capacity=0, scores=True, stats=False, workspace=None, stream=None):
    """Packed variable-length batch: sequence b owns queries cu_q[b]:cu_q[b+1]
    and keys cu_k[b]:cu_k[b+1]; positions and returned indices are relative to
    the sequence. Same outputs as :func:`select` over the concatenated rows."""
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    _check_tensor("positions", positions, dev, torch.int32, (n,))
    cq, ck = _offsets(cu_q, "cu_q"), _offsets(cu_k, "cu_k")
    if cq.size != ck.size or cq[-1] != n or ck[-1] != L:
        raise ValueError("cu_q / cu_k do not match the query and key counts")
    B = cq.size - 1
    idx = torch.empty((n, k_top), dtype=torch.int32, device=dev)
    sc = torch.empty((n, k_top), dtype=torch.float32, device=dev) if scores else None
    need = lib.hytopk_select_varlen_workspace_size(_cu_ptr(cq), _cu_ptr(ck), B, H, d, k_top,
                                                   capacity, dt)
    if need == 0:
        raise HytopkError(2, "hytopk_select_varlen_workspace_size")
    ws = _workspace(need, dev, workspace)
    st = torch.zeros(8, dtype=torch.int32, device=dev) if stats else None
    status = lib.hytopk_select_varlen(
        _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(positions), _cu_ptr(cq),
        _cu_ptr(ck), B, H, d, k_top, dt, _ptr(idx), _ptr(sc), capacity, _ptr(ws), ws.numel(),
        _ptr(st), _stream(dev, stream))
    if status != 0:
        raise HytopkError(status, "hytopk_select_varlen")
    return idx, sc, st


def replay_varlen(q, k, w, idx, cu_q, cu_k, *, q_scale=None, k_scale=None, status=None,
                  stream=None):
    """Selection replay over a packed variable-length batch (indices relative
    to each query's sequence)."""
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    k_top = idx.shape[1]
    _check_tensor("idx", idx, dev, torch.int32, (n, k_top))
    cq, ck = _offsets(cu_q, "cu_q"), _offsets(cu_k, "cu_k")
    if cq.size != ck.size or cq[-1] != n or ck[-1] != L:
        raise ValueError("cu_q / cu_k do not match the query and key counts")
    res = torch.empty((n, k_top), dtype=torch.float32, device=dev)
    st = lib.hytopk_replay_varlen(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                                  _ptr(idx), _cu_ptr(cq), _cu_ptr(ck), cq.size - 1, H, d, k_top,
                                  dt, _ptr(res), _ptr(status), _stream(dev, stream))
    if st != 0:
        raise HytopkError(st, "hytopk_replay_varlen")
    return res


def replay_backward_varlen(q, k, w, idx, grad, cu_q, cu_k, *, q_scale=None, k_scale=None,
                           dk=None, status=None, stream=None):
    """Gradients at the selected entries of a packed variable-length batch
    (indices relative to each query's sequence): (dq, dk, dw) as
    :func:`replay_backward`; dk covers all sequences' keys and is added to."""
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    k_top = idx.shape[1]
    _check_tensor("idx", idx, dev, torch.int32, (n, k_top))
    _check_tensor("grad", grad, dev, torch.float32, (n, k_top))
    cq, ck = _offsets(cu_q, "cu_q"), _offsets(cu_k, "cu_k")
    if cq.size != ck.size or cq[-1] != n or ck[-1] != L:
        raise ValueError("cu_q / cu_k do not match the query and key counts")
    dq = torch.empty((n, H, d), dtype=torch.float32, device=dev)
    dw = torch.empty((n, H), dtype=torch.float32, device=dev)
    if dk is None:
        dk = torch.zeros((L, d), dtype=torch.float32, device=dev)
    else:
        _check_tensor("dk", dk, dev, torch.float32, (L, d))
    st = lib.hytopk_replay_backward_varlen(
        _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(idx), _ptr(grad),
        _cu_ptr(cq), _cu_ptr(ck), cq.size - 1, H, d, k_top, dt, _ptr(dq), _ptr(dk), _ptr(dw),
        _ptr(status), _stream(dev, stream))
    if st != 0:
        raise HytopkError(st, "hytopk_replay_backward_varlen")
    return dq, dk, dw


def read_stats(st) -> dict:
    """Decode a stats tensor returned by :func:`select` (synchronises)."""
    raw = st.cpu().numpy().tobytes()
    s = Stats.from_buffer_copy(raw[:ctypes.sizeof(Stats)])
    return {name: getattr(s, name) for name, _ in Stats._fields_}


def replay(q, k, w, idx, *, q_scale=None, k_scale=None, status=None, out=None, group=1,
           stream=None):
    """Selection replay: scores [n,k] of the stored indices idx [n,k].
    ``group=2`` replays adjacent query pairs over the union of their indices
    (same result)."""
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    k_top = idx.shape[1]
    _check_tensor("idx", idx, dev, torch.int32, (n, k_top))
    res = out if out is not None else torch.empty((n, k_top), dtype=torch.float32, device=dev)
    if group == 1:
        st = lib.hytopk_replay(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(idx),
                               n, L, H, d, k_top, dt, _ptr(res), _ptr(status),
                               _stream(dev, stream))
    else:
        st = lib.hytopk_replay_grouped(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                                       _ptr(idx), n, L, H, d, k_top, dt, group, _ptr(res),
                                       _ptr(status), _stream(dev, stream))
    if st != 0:
        raise HytopkError(st, "hytopk_replay")
    return res


def replay_backward(q, k, w, idx, grad, *, q_scale=None, k_scale=None, dk=None, status=None,
                    stream=None):
    """Gradients at the selected entries: returns (dq [n,H,d], dk [L,d], dw [n,H]),
    fp32. ``dk`` is added to when given (else a zeroed tensor is used)."""
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    k_top = idx.shape[1]
    _check_tensor("idx", idx, dev, torch.int32, (n, k_top))
    _check_tensor("grad", grad, dev, torch.float32, (n, k_top))
    dq = torch.empty((n, H, d), dtype=torch.float32, device=dev)
    dw = torch.empty((n, H), dtype=torch.float32, device=dev)
    if dk is None:
        dk = torch.zeros((L, d), dtype=torch.float32, device=dev)
    else:
        _check_tensor("dk", dk, dev, torch.float32, (L, d))
    st = lib.hytopk_replay_backward(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                                    _ptr(idx), _ptr(grad), n, L, H, d, k_top, dt, _ptr(dq),
                                    _ptr(dk), _ptr(dw), _ptr(status), _stream(dev, stream))
    if st != 0:
        raise HytopkError(st, "hytopk_replay_backward")
    return dq, dk, dw


def select_twopass(q, k, w, positions, k_top, *, q_scale=None, k_scale=None, rows_per_chunk=0,
                   scores=True, workspace=None, status=None, stream=None):
    """The conventional materialise-then-top-k path (same outputs as select)."""
    import torch

    lib = load()
    dt, n, L, H, d, dev = _common(q, q_scale, k, k_scale, w)
    _check_tensor("positions", positions, dev, torch.int32, (n,))
    idx = torch.empty((n, k_top), dtype=torch.int32, device=dev)
    sc = torch.empty((n, k_top), dtype=torch.float32, device=dev) if scores else None
    # with a caller workspace the library picks the largest chunk that fits
    need = lib.hytopk_twopass_workspace_size(n, L, H, d, k_top, dt,
                                             1 if workspace is not None else rows_per_chunk)
    if need == 0:
        raise HytopkError(2, "hytopk_twopass_workspace_size")
    ws = _workspace(need, dev, workspace)
    st = lib.hytopk_select_twopass(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w),
                                   _ptr(positions), n, L, H, d, k_top, dt, _ptr(idx), _ptr(sc),
                                   _ptr(ws), ws.numel(), _ptr(status), _stream(dev, stream))
    if st != 0:
        raise HytopkError(st, "hytopk_select_twopass")
    return idx, sc


# ---- around the selection: rotary positions, cache rows, attention ------------------
# These calls also serve single tokens, where the time is the host's, so their checks,
# allocations and calls are in a C++ module (csrc/binding.cpp). They are not recorded by
# autograd; with ``stream=`` their results come from that stream's memory.

_module = None


def _operators():
    """The operators' module, loaded once (raises if it has not been built)."""
    global _module
    if _module is None:
        import importlib.machinery
        import importlib.util

        import torch

        lib = load()
        path = _build.binding()
        if not os.path.exists(path):
            raise RuntimeError(f"the operators' module is not built ({path}); "
                               "call exact_top_token_gb300.build() first")
        loader = importlib.machinery.ExtensionFileLoader("_operators", path)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location("_operators", path, loader=loader))
        loader.exec_module(module)
        module.init(HytopkError, torch.OutOfMemoryError, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.hytopk_rope, lib.hytopk_cache_write, lib.hytopk_cache_read, lib.hytopk_attend,
            lib.hytopk_attend_backward)))
        _module = module
    return _module


def rope_frequencies(rot, base=10000.0, *, scaling=None, factor=1.0, original_context=None,
                     fast=32.0, slow=1.0, device="cuda"):
    """(inv_freq [rot/2] fp32 tensor, mscale): the frequency table of ``rot``
    rotated columns, base ** (-2 i / rot), and the factor that goes with it, to be
    given to :func:`rope` and :func:`cache_write` for queries and keys alike.

    ``scaling`` stretches it for contexts ``factor`` times the original one:
    ``None``; ``"linear"`` (all frequencies divided by the factor); ``"base"``
    (the base raised to base * factor ** (rot / (rot - 2)), which keeps the
    highest frequency and divides the lowest by the factor); ``"parts"``
    (frequencies that turn more than ``fast`` times within
    ``original_context`` are kept, those below ``slow`` turns divided by the
    factor, a linear ramp over the turns between; mscale = 0.1 ln(factor) + 1).
    A table made another way (a ramp over the column, say) goes to :func:`rope` as it is.
    """
    import math

    import torch

    if rot < 2 or rot % 2 or not base > 0 or not factor >= 1.0:
        raise ValueError("rot must be even and positive, base positive, factor at least 1")
    mscale = 1.0
    if scaling == "base":
        if rot < 4:
            raise ValueError("base scaling needs at least two pairs")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not original_context or original_context < 1 or not fast > slow:
            raise ValueError("parts scaling needs original_context and fast > slow")
        turns = original_context * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.float().to(device), mscale


def rope(x, positions, inv_freq, *, first=0, interleaved=False, mscale=1.0, inverse=False,
         out=None, status=None, stream=None):
    """Rotary positions on columns [first, first + 2 len(inv_freq)) of x
    ([n, H, d] or [n, d], bf16 or fp32, row and head strides allowed); the
    other columns are copied. Pairs are (i, i + rot/2), or (2i, 2i + 1) if
    ``interleaved``. ``out=x`` works in place. ``inverse`` rotates back, which
    is also the gradient. See :func:`rope_frequencies`."""
    return (_module or _operators()).rope(x, positions, inv_freq, first, interleaved, mscale,
                                          inverse, out, status, stream)


def cache_write(x, cache, cache_scale=None, *, slots=None, positions=None, inv_freq=None, first=0,
                interleaved=False, mscale=1.0, status=None, stream=None):
    """Write rows x ([n, H, d] or [n, d], bf16 or fp32) into cache rows
    ``slots`` (int32 [n], -1 skips; None: rows 0..n-1), rotated first when
    ``positions`` and ``inv_freq`` are given, and quantised when the cache
    ([L, H, d] or [L, d]) is float8_e4m3fn: one scale per (row, head) in
    ``cache_scale``, as :func:`select` and :func:`attend` take them."""
    return (_module or _operators()).cache_write(x, cache, cache_scale, slots, positions, inv_freq,
                                                 first, interleaved, mscale, status, stream)


def cache_read(cache, cache_scale=None, *, slots=None, dtype=None, out=None, status=None,
               stream=None):
    """Cache rows ``slots`` (int32 [m]; None: all) as bf16 (default) or fp32."""
    return (_module or _operators()).cache_read(cache, cache_scale, slots, dtype, out, status,
                                                stream)


def attend(q, k, v, idx, *, k_scale=None, v_scale=None, scale=None, out_dtype=None, out=None,
           status=None, stream=None):
    """Attention of each query over its own selected rows: q [n, Hq, d] bf16,
    k and v [L, Hkv, d] (or [L, d]) bf16 or float8_e4m3fn with k_scale /
    v_scale [L, Hkv] (or [L]) fp32, idx [n, k] int32 as :func:`select` returns
    it (-1: none). ``scale`` defaults to d ** -0.5. Returns ``(out [n, Hq, d],
    lse [n, Hq])``; ``out_dtype`` bf16 (default) or fp32 (for training:
    :func:`attend_backward` then keeps fp32 accuracy)."""
    return (_module or _operators()).attend(q, k, v, idx, k_scale, v_scale, scale, out_dtype, out,
                                            status, stream)


def attend_backward(q, k, v, idx, out, lse, grad, *, scale=None, dk=None, dv=None, status=None,
                    stream=None):
    """Gradients of :func:`attend` (bf16 k and v): ``(dq [n, Hq, d], dk, dv)``
    in fp32, dk and dv shaped like k. ``grad`` [n, Hq, d] bf16 is the gradient
    of out. ``dk`` and ``dv`` are added to when given (both or neither; else new
    tensors are written)."""
    return (_module or _operators()).attend_backward(q, k, v, idx, out, lse, grad, scale, dk, dv,
                                                     status, stream)
