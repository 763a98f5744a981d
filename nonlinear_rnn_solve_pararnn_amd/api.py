"""Thin Python binding of libpararnn.so (include/pararnn.h).

Argument marshalling only: checks dtype, device, shape and contiguity,
allocates outputs and the workspace with torch (the caching allocator, so no
hipMalloc per call), passes raw device pointers and the current HIP stream to
the C ABI, and raises on a negative status.  Every step of the computation
runs in the library's HIP kernels; there is no fallback of any kind, and a
missing library raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
import weakref
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpararnn.so")

OP_LINSCAN_DIAG, OP_LINSCAN_BLK2, OP_GRU_FORWARD, OP_LSTM_FORWARD, OP_GRU_ADJOINT, \
    OP_LSTM_ADJOINT, OP_LINSCAN_BLK4, OP_LINSCAN_BLK8, OP_HGRU4_FORWARD, OP_HGRU8_FORWARD, \
    OP_HGRU4_BACKWARD, OP_HGRU8_BACKWARD = range(12)
CELL_GRU, CELL_LSTM = 0, 1

EXPORTS = ("pararnn_workspace_bytes", "rnn_linscan_diag", "rnn_linscan_blk2", "rnn_linscan_blk",
           "pararnn_gru_forward", "pararnn_lstm_forward", "pararnn_adjoint_backward",
           "pararnn_gru_sequential", "pararnn_lstm_sequential", "pararnn_status_string",
           "pararnn_gru_forward_noalloc", "pararnn_hgru_forward", "pararnn_hgru_backward",
           "pararnn_linattn_workspace_bytes", "pararnn_linattn_forward", "pararnn_linattn_backward",
           "pararnn_linattn_step", "pararnn_layernorm_workspace_bytes", "pararnn_layernorm_forward",
           "pararnn_layernorm_backward", "pararnn_embedding_forward",
           "pararnn_embedding_workspace_bytes", "pararnn_embedding_backward")
NOALLOC_SCRATCH_BYTES = 64 << 20   # PARARNN_NOALLOC_SCRATCH_BYTES

_lib = None


class PararnnError(RuntimeError):
    pass


def load_library():
    """Load libpararnn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise PararnnError(
            "libpararnn.so not found at %s; build it with "
            "`python -m nonlinear_rnn_solve_pararnn_amd.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    sz = ctypes.c_size_t
    lib.pararnn_workspace_bytes.argtypes = [i32, i64, i64, i64, i32]
    lib.pararnn_workspace_bytes.restype = sz
    lib.rnn_linscan_diag.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.rnn_linscan_diag.restype = ctypes.c_int
    lib.rnn_linscan_blk2.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.rnn_linscan_blk2.restype = ctypes.c_int
    lib.rnn_linscan_blk.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.rnn_linscan_blk.restype = ctypes.c_int
    lib.pararnn_gru_forward.argtypes = [i64, i64, i64] + [vp] * 9 + [
        ctypes.c_float, i32, vp, vp, vp, sz, vp]
    lib.pararnn_gru_forward.restype = ctypes.c_int
    lib.pararnn_lstm_forward.argtypes = [i64, i64, i64] + [vp] * 14 + [
        ctypes.c_float, i32, vp, vp, vp, sz, vp]
    lib.pararnn_lstm_forward.restype = ctypes.c_int
    lib.pararnn_hgru_forward.argtypes = [i32, i64, i64, i64] + [vp] * 9 + [
        ctypes.c_float, i32, vp, vp, vp, sz, vp]
    lib.pararnn_hgru_forward.restype = ctypes.c_int
    lib.pararnn_hgru_backward.argtypes = [i32, i64, i64, i64] + [vp] * 17 + [sz, vp]
    lib.pararnn_hgru_backward.restype = ctypes.c_int
    lib.pararnn_adjoint_backward.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                             vp, vp, vp, vp, vp, sz, vp]
    lib.pararnn_adjoint_backward.restype = ctypes.c_int
    lib.pararnn_gru_sequential.argtypes = [i64, i64, i64] + [vp] * 8 + [vp]
    lib.pararnn_gru_sequential.restype = ctypes.c_int
    lib.pararnn_lstm_sequential.argtypes = [i64, i64, i64] + [vp] * 12 + [vp]
    lib.pararnn_lstm_sequential.restype = ctypes.c_int
    lib.pararnn_gru_forward_noalloc.argtypes = [i64, i64, i64] + [vp] * 8 + [
        ctypes.c_float, i32, vp, vp, vp]
    lib.pararnn_gru_forward_noalloc.restype = ctypes.c_int
    lib.pararnn_linattn_workspace_bytes.argtypes = [i32, i32] + [i64] * 5
    lib.pararnn_linattn_workspace_bytes.restype = sz
    lib.pararnn_linattn_forward.argtypes = [i32] + [i64] * 5 + [vp] * 6 + [
        ctypes.c_float, vp, vp, vp, sz, vp]
    lib.pararnn_linattn_forward.restype = ctypes.c_int
    lib.pararnn_linattn_backward.argtypes = [i32] + [i64] * 5 + [vp] * 8 + [
        ctypes.c_float, vp, vp, vp, vp, vp, sz, vp]
    lib.pararnn_linattn_backward.restype = ctypes.c_int
    lib.pararnn_linattn_step.argtypes = [i32] + [i64] * 4 + [vp] * 6 + [ctypes.c_float, vp, vp, vp]
    lib.pararnn_linattn_step.restype = ctypes.c_int
    lib.pararnn_layernorm_workspace_bytes.argtypes = [i64, i64]
    lib.pararnn_layernorm_workspace_bytes.restype = sz
    lib.pararnn_layernorm_forward.argtypes = [i32, i64, i64] + [vp] * 4 + [ctypes.c_float] + [vp] * 5
    lib.pararnn_layernorm_forward.restype = ctypes.c_int
    lib.pararnn_layernorm_backward.argtypes = [i32, i64, i64] + [vp] * 10 + [sz, vp]
    lib.pararnn_layernorm_backward.restype = ctypes.c_int
    lib.pararnn_embedding_forward.argtypes = [i32, i64, i64, i64, vp, i32, vp, ctypes.c_float, vp, vp]
    lib.pararnn_embedding_forward.restype = ctypes.c_int
    lib.pararnn_embedding_workspace_bytes.argtypes = [i64, i64, i64]
    lib.pararnn_embedding_workspace_bytes.restype = sz
    lib.pararnn_embedding_backward.argtypes = [i32, i64, i64, i64, vp, i32, vp, ctypes.c_float, i64,
                                               vp, vp, sz, vp]
    lib.pararnn_embedding_backward.restype = ctypes.c_int
    lib.pararnn_status_string.argtypes = [ctypes.c_int]
    lib.pararnn_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        msg = load_library().pararnn_status_string(status).decode()
        raise PararnnError("%s failed: status %d (%s)" % (what, status, msg))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(_raw_stream(device))


def _need(t: torch.Tensor, shape, name: str, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != torch.float32:
        raise TypeError("%s must be float32, got %s" % (name, t.dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be on a HIP device" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def workspace_bytes(op: int, B: int, L: int, H: int, max_iter: int = 1) -> int:
    return int(load_library().pararnn_workspace_bytes(op, B, L, H, max_iter))


# One zero-filled workspace per (device, stream, host thread), grown on demand.
# The library leaves a workspace ready for the next call of any entry point, so
# it is cleared only when it is first allocated.  Threads have their own: two
# that issue on one stream may interleave the launches of their calls.  A
# thread's go when it ends.
class _Kept(dict):
    __hash__ = object.__hash__


class _Thread(threading.local):
    def __init__(self):
        self.kept = _Kept()
        _all_kept.add(self.kept)


_all_kept = weakref.WeakSet()
_thread = _Thread()
_WS_HEADER = 256   # bytes before an operator's scratch: a call that needs no more uses none of them


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled workspace of at least `nbytes` bytes (the library requires
    a zero-filled workspace on first use; later calls keep it valid)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def release_workspaces():
    """Drop the cached workspaces."""
    for kept in list(_all_kept):
        kept.clear()


def _workspace(op, B, L, H, device, max_iter=1, ws=None):
    n = workspace_bytes(op, B, L, H, max_iter)
    if n == 0:
        raise PararnnError("invalid sizes B=%d L=%d H=%d" % (B, L, H))
    return _workspace_of(n, device, ws)


def _raw_stream(device: torch.device) -> int:
    """The device's current HIP stream as an integer (a stream object costs more than a small kernel's launch)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _capturing() -> bool:
    """Whether the current stream's calls go into a HIP graph."""
    return torch._C._cuda_isCurrentStreamCapturing()


@functools.lru_cache(maxsize=None)
def _no_scratch(device: torch.device) -> torch.Tensor:
    """What calls that use no scratch are given: never read nor written."""
    return new_workspace(_WS_HEADER, device)


def _workspace_of(n: int, device, ws=None, scratch=False):
    """The caller's workspace if one is given, else the one this thread keeps for
    the stream, of at least n bytes.  A call that is being captured gets one of its
    own from the graph's memory (cleared in the graph, unless it is only scratch):
    replays must not depend on a buffer that a later call may replace or use."""
    if ws is not None:
        if ws.device != device or ws.numel() * ws.element_size() < n or ws.data_ptr() % 256:
            raise ValueError("workspace too small, misaligned or on the wrong device")
        return ws, ws.numel() * ws.element_size()
    if scratch and n <= _WS_HEADER:
        return _no_scratch(device), _WS_HEADER
    if _capturing():
        buf = torch.empty(max(n, 256), dtype=torch.uint8, device=device) if scratch else new_workspace(n, device)
        return buf, buf.numel()
    kept, key = _thread.kept, (device.index, _raw_stream(device))
    buf = kept.get(key)
    if buf is None or buf.numel() < n:
        buf = new_workspace(n, device)
        kept[key] = buf
    return buf, buf.numel()


# ---------------------------------------------------------------- scans
def linscan_diag(a, b, h0=None, *, out=None, ws=None):
    """h_t = a_t * h_{t-1} + b_t over dim 1 of [B, L, H] tensors."""
    lib = load_library()
    B, L, H = a.shape
    dev = a.device
    _need(a, (B, L, H), "a")
    _need(b, (B, L, H), "b", dev)
    if h0 is not None:
        _need(h0, (B, H), "h0", dev)
    h = torch.empty_like(a) if out is None else out
    _need(h, (B, L, H), "out", dev)
    ws, n = _workspace(OP_LINSCAN_DIAG, B, L, H, dev, ws=ws)
    _check(lib.rnn_linscan_diag(B, L, H, _ptr(a), _ptr(b), _ptr(h0), _ptr(h), _ptr(ws), n,
                                _stream(dev)), "rnn_linscan_diag")
    return h


def linscan_blk2(A, b, h0=None, *, out=None, ws=None):
    """h_t = A_t @ h_{t-1} + b_t with A [B, L, H, 2, 2], b/h [B, L, H, 2]."""
    lib = load_library()
    B, L, H = b.shape[:3]
    dev = b.device
    _need(A, (B, L, H, 2, 2), "A", dev)
    _need(b, (B, L, H, 2), "b", dev)
    if h0 is not None:
        _need(h0, (B, H, 2), "h0", dev)
    h = torch.empty_like(b) if out is None else out
    _need(h, (B, L, H, 2), "out", dev)
    ws, n = _workspace(OP_LINSCAN_BLK2, B, L, H, dev, ws=ws)
    _check(lib.rnn_linscan_blk2(B, L, H, _ptr(A), _ptr(b), _ptr(h0), _ptr(h), _ptr(ws), n,
                                _stream(dev)), "rnn_linscan_blk2")
    return h


# ---------------------------------------------------------------- Newton forward
def linscan_blk(A, b, h0=None, *, out=None, ws=None):
    """k x k block scan h_t = A_t h_{t-1} + b_t (k = 2, 4 or 8); A [B, L, H, k, k],
    b [B, L, H, k]; returns h [B, L, H, k]."""
    lib = load_library()
    B, L, H, k = b.shape
    dev = b.device
    _need(A, (B, L, H, k, k), "A", dev)
    _need(b, (B, L, H, k), "b", dev)
    if h0 is not None:
        _need(h0, (B, H, k), "h0", dev)
    h = torch.empty_like(b) if out is None else out
    _need(h, (B, L, H, k), "out", dev)
    op = {2: OP_LINSCAN_BLK2, 4: OP_LINSCAN_BLK4, 8: OP_LINSCAN_BLK8}.get(k)
    if op is None:
        raise PararnnError("rnn_linscan_blk supports k = 2, 4 and 8, got %d" % k)
    ws, n = _workspace(op, B, L, H, dev, ws=ws)
    _check(lib.rnn_linscan_blk(k, B, L, H, _ptr(A), _ptr(b), _ptr(h0), _ptr(h), _ptr(ws), n,
                               _stream(dev)), "rnn_linscan_blk")
    return h


def gru_forward(pz, pr, pc, uz, ur, uc, h0=None, *, tol=1e-4, max_iter=32, out=None,
                info=None, trace=None, ws=None, init=None):
    """Newton solve of the diagonal GRU over [B, L, H] gate pre-projections.

    Returns h [B, L, H].  `init` [B, L, H] is Newton's initial iterate (a warm
    start; None starts from zero; it must not share memory with the output).
    `info` (int32[2] device tensor) receives {iterations, converged}; `trace`
    (float32[max_iter]) receives max|delta| per iteration."""
    lib = load_library()
    B, L, H = pz.shape
    dev = pz.device
    for t, n in ((pz, "pz"), (pr, "pr"), (pc, "pc")):
        _need(t, (B, L, H), n, dev)
    for t, n in ((uz, "uz"), (ur, "ur"), (uc, "uc")):
        _need(t, (H,), n, dev)
    if h0 is not None:
        _need(h0, (B, H), "h0", dev)
    if init is not None:
        _need(init, (B, L, H), "init", dev)
    h = torch.empty_like(pz) if out is None else out
    _need(h, (B, L, H), "out", dev)
    if info is not None and (info.dtype != torch.int32 or info.numel() < 2 or info.device != dev):
        raise ValueError("info must be an int32 device tensor with 2 elements")
    if trace is not None and (trace.dtype != torch.float32 or trace.numel() < max_iter or
                              trace.device != dev):
        raise ValueError("trace must be a float32 device tensor with max_iter elements")
    ws, n = _workspace(OP_GRU_FORWARD, B, L, H, dev, max_iter, ws)
    _check(lib.pararnn_gru_forward(B, L, H, _ptr(pz), _ptr(pr), _ptr(pc), _ptr(uz), _ptr(ur),
                                   _ptr(uc), _ptr(h0), _ptr(init), _ptr(h), float(tol),
                                   int(max_iter), _ptr(info), _ptr(trace), _ptr(ws), n,
                                   _stream(dev)),
           "pararnn_gru_forward")
    return h


def lstm_forward(pi, pf, po, pg, ui, uf, uo, ug, h0=None, c0=None, *, tol=1e-4, max_iter=32,
                 out_h=None, out_c=None, info=None, trace=None, ws=None, init_h=None,
                 init_c=None):
    """Newton solve of the diagonal LSTM; returns (h, c), each [B, L, H].
    `init_h`, `init_c` [B, L, H]: Newton's initial iterates (a warm start; a
    missing one is zero; neither may share memory with the outputs)."""
    lib = load_library()
    B, L, H = pi.shape
    dev = pi.device
    for t, n in ((pi, "pi"), (pf, "pf"), (po, "po"), (pg, "pg")):
        _need(t, (B, L, H), n, dev)
    for t, n in ((ui, "ui"), (uf, "uf"), (uo, "uo"), (ug, "ug")):
        _need(t, (H,), n, dev)
    if h0 is not None:
        _need(h0, (B, H), "h0", dev)
    if c0 is not None:
        _need(c0, (B, H), "c0", dev)
    if init_h is not None:
        _need(init_h, (B, L, H), "init_h", dev)
    if init_c is not None:
        _need(init_c, (B, L, H), "init_c", dev)
    h = torch.empty_like(pi) if out_h is None else out_h
    c = torch.empty_like(pi) if out_c is None else out_c
    _need(h, (B, L, H), "out_h", dev)
    _need(c, (B, L, H), "out_c", dev)
    if info is not None and (info.dtype != torch.int32 or info.numel() < 2 or info.device != dev):
        raise ValueError("info must be an int32 device tensor with 2 elements")
    if trace is not None and (trace.dtype != torch.float32 or trace.numel() < max_iter or
                              trace.device != dev):
        raise ValueError("trace must be a float32 device tensor with max_iter elements")
    ws, n = _workspace(OP_LSTM_FORWARD, B, L, H, dev, max_iter, ws)
    _check(lib.pararnn_lstm_forward(B, L, H, _ptr(pi), _ptr(pf), _ptr(po), _ptr(pg), _ptr(ui),
                                    _ptr(uf), _ptr(uo), _ptr(ug), _ptr(h0), _ptr(c0),
                                    _ptr(init_h), _ptr(init_c), _ptr(h), _ptr(c), float(tol),
                                    int(max_iter), _ptr(info), _ptr(trace), _ptr(ws), n,
                                    _stream(dev)), "pararnn_lstm_forward")
    return h, c


def hgru_forward(pz, pr, pc, Uz, Ur, Uc, h0=None, *, tol=1e-4, max_iter=32, out=None, info=None,
                 trace=None, ws=None, init=None):
    """Newton solve of the GRU with dense recurrence inside heads of k
    channels (k = 4 or 8): p [B, L, NH, k], U [NH, k, k], h0 [B, NH, k];
    returns h [B, L, NH, k].  `init` is Newton's initial iterate (a warm
    start; it must not share memory with the output); `info`, `trace` as for
    gru_forward."""
    lib = load_library()
    B, L, NH, k = pz.shape
    dev = pz.device
    for t, n in ((pz, "pz"), (pr, "pr"), (pc, "pc")):
        _need(t, (B, L, NH, k), n, dev)
    for t, n in ((Uz, "Uz"), (Ur, "Ur"), (Uc, "Uc")):
        _need(t, (NH, k, k), n, dev)
    if h0 is not None:
        _need(h0, (B, NH, k), "h0", dev)
    if init is not None:
        _need(init, (B, L, NH, k), "init", dev)
    op = {4: OP_HGRU4_FORWARD, 8: OP_HGRU8_FORWARD}.get(k)
    if op is None:
        raise PararnnError("pararnn_hgru_forward supports k = 4 and 8, got %d" % k)
    h = torch.empty_like(pz) if out is None else out
    _need(h, (B, L, NH, k), "out", dev)
    if info is not None and (info.dtype != torch.int32 or info.numel() < 2 or info.device != dev):
        raise ValueError("info must be an int32 device tensor with 2 elements")
    if trace is not None and (trace.dtype != torch.float32 or trace.numel() < max_iter or
                              trace.device != dev):
        raise ValueError("trace must be a float32 device tensor with max_iter elements")
    ws, n = _workspace(op, B, L, NH, dev, max_iter, ws)
    _check(lib.pararnn_hgru_forward(k, B, L, NH, _ptr(pz), _ptr(pr), _ptr(pc), _ptr(Uz), _ptr(Ur),
                                    _ptr(Uc), _ptr(h0), _ptr(init), _ptr(h), float(tol), int(max_iter),
                                    _ptr(info), _ptr(trace), _ptr(ws), n, _stream(dev)),
           "pararnn_hgru_forward")
    return h


def hgru_backward(pz, pr, pc, Uz, Ur, Uc, h0, h, grad_h, *, want_u=True, want_h0=True, ws=None, out=None):
    """Gradients of sum(grad_h * h) through the head-GRU solve h (the
    converged output of hgru_forward): returns (dpz, dpr, dpc, dUz, dUr, dUc,
    dh0), the U gradients None unless want_u, dh0 None unless want_h0.
    `out`: the seven output tensors to write instead (None entries for the
    gradients not wanted)."""
    lib = load_library()
    B, L, NH, k = pz.shape
    dev = pz.device
    for t, n in ((pz, "pz"), (pr, "pr"), (pc, "pc"), (h, "h"), (grad_h, "grad_h")):
        _need(t, (B, L, NH, k), n, dev)
    for t, n in ((Uz, "Uz"), (Ur, "Ur"), (Uc, "Uc")):
        _need(t, (NH, k, k), n, dev)
    if h0 is not None:
        _need(h0, (B, NH, k), "h0", dev)
    op = {4: OP_HGRU4_BACKWARD, 8: OP_HGRU8_BACKWARD}.get(k)
    if op is None:
        raise PararnnError("pararnn_hgru_backward supports k = 4 and 8, got %d" % k)
    if out is not None:
        gp, gU, gh0 = list(out[:3]), list(out[3:6]), out[6]
        for t, n in zip(gp, ("dpz", "dpr", "dpc")):
            _need(t, (B, L, NH, k), n, dev)
        for t, n in zip(gU, ("dUz", "dUr", "dUc")):
            if t is not None:
                _need(t, (NH, k, k), n, dev)
        if gh0 is not None:
            _need(gh0, (B, NH, k), "dh0", dev)
    else:
        gp = [torch.empty_like(pz) for _ in range(3)]
        gU = [torch.empty_like(Uz) for _ in range(3)] if want_u else [None] * 3
        gh0 = torch.empty(B, NH, k, device=dev) if want_h0 else None
    ws, n = _workspace(op, B, L, NH, dev, 1, ws)
    _check(lib.pararnn_hgru_backward(k, B, L, NH, _ptr(pz), _ptr(pr), _ptr(pc), _ptr(Uz), _ptr(Ur), _ptr(Uc),
                                     _ptr(h0), _ptr(h), _ptr(grad_h), _ptr(gp[0]), _ptr(gp[1]), _ptr(gp[2]),
                                     _ptr(gU[0]), _ptr(gU[1]), _ptr(gU[2]), _ptr(gh0), _ptr(ws), n, _stream(dev)),
           "pararnn_hgru_backward")
    return (*gp, *gU, gh0)


def gru_forward_noalloc(pz, pr, pc, uz, ur, uc, h0=None, *, tol=1e-4, max_iter=32, out=None,
                        info=None, trace=None):
    """gru_forward with the library's static scratch buffer as workspace
    (pararnn_gru_forward_noalloc): the call allocates nothing on the device
    when `out` is given."""
    lib = load_library()
    B, L, H = pz.shape
    dev = pz.device
    for t, n in ((pz, "pz"), (pr, "pr"), (pc, "pc")):
        _need(t, (B, L, H), n, dev)
    for t, n in ((uz, "uz"), (ur, "ur"), (uc, "uc")):
        _need(t, (H,), n, dev)
    if h0 is not None:
        _need(h0, (B, H), "h0", dev)
    h = torch.empty_like(pz) if out is None else out
    _need(h, (B, L, H), "out", dev)
    if info is not None and (info.dtype != torch.int32 or info.numel() < 2 or info.device != dev):
        raise ValueError("info must be an int32 device tensor with 2 elements")
    if trace is not None and (trace.dtype != torch.float32 or trace.numel() < max_iter or
                              trace.device != dev):
        raise ValueError("trace must be a float32 device tensor with max_iter elements")
    _check(lib.pararnn_gru_forward_noalloc(B, L, H, _ptr(pz), _ptr(pr), _ptr(pc), _ptr(uz), _ptr(ur),
                                           _ptr(uc), _ptr(h0), _ptr(h), float(tol), int(max_iter),
                                           _ptr(info), _ptr(trace), _stream(dev)),
           "pararnn_gru_forward_noalloc")
    return h


# ---------------------------------------------------------------- sequential
def gru_sequential(pz, pr, pc, uz, ur, uc, h0=None, *, out=None):
    """Sequential application of the GRU cell (one thread per channel, one
    cell per position); returns h [B, L, H]."""
    lib = load_library()
    B, L, H = pz.shape
    dev = pz.device
    for t, n in ((pz, "pz"), (pr, "pr"), (pc, "pc")):
        _need(t, (B, L, H), n, dev)
    for t, n in ((uz, "uz"), (ur, "ur"), (uc, "uc")):
        _need(t, (H,), n, dev)
    if h0 is not None:
        _need(h0, (B, H), "h0", dev)
    h = torch.empty_like(pz) if out is None else out
    _need(h, (B, L, H), "out", dev)
    _check(lib.pararnn_gru_sequential(B, L, H, _ptr(pz), _ptr(pr), _ptr(pc), _ptr(uz), _ptr(ur),
                                      _ptr(uc), _ptr(h0), _ptr(h), _stream(dev)),
           "pararnn_gru_sequential")
    return h


def lstm_sequential(pi, pf, po, pg, ui, uf, uo, ug, h0=None, c0=None, *, out_h=None, out_c=None):
    """Sequential application of the LSTM cell; returns (h, c), each [B, L, H]."""
    lib = load_library()
    B, L, H = pi.shape
    dev = pi.device
    for t, n in ((pi, "pi"), (pf, "pf"), (po, "po"), (pg, "pg")):
        _need(t, (B, L, H), n, dev)
    for t, n in ((ui, "ui"), (uf, "uf"), (uo, "uo"), (ug, "ug")):
        _need(t, (H,), n, dev)
    if h0 is not None:
        _need(h0, (B, H), "h0", dev)
    if c0 is not None:
        _need(c0, (B, H), "c0", dev)
    h = torch.empty_like(pi) if out_h is None else out_h
    c = torch.empty_like(pi) if out_c is None else out_c
    _need(h, (B, L, H), "out_h", dev)
    _need(c, (B, L, H), "out_c", dev)
    _check(lib.pararnn_lstm_sequential(B, L, H, _ptr(pi), _ptr(pf), _ptr(po), _ptr(pg), _ptr(ui),
                                       _ptr(uf), _ptr(uo), _ptr(ug), _ptr(h0), _ptr(c0), _ptr(h),
                                       _ptr(c), _stream(dev)), "pararnn_lstm_sequential")
    return h, c


# ---------------------------------------------------------------- adjoint
def adjoint_backward(cell: int, p: Sequence[torch.Tensor], u: Sequence[torch.Tensor],
                     h: torch.Tensor, grad_h: torch.Tensor, h0=None, *, c=None, c0=None,
                     grad_c=None, want_u=True, want_h0=True, want_c0=True, ws=None):
    """Reverse-time adjoint of the converged solve.  Returns a dict with
    'p' (list of [B, L, H]), 'u' (list of [H] or None), 'h0', 'c0'."""
    lib = load_library()
    ng = 3 if cell == CELL_GRU else 4
    if len(p) != ng or len(u) != ng:
        raise ValueError("expected %d gate tensors" % ng)
    B, L, H = h.shape
    dev = h.device
    for k, t in enumerate(p):
        _need(t, (B, L, H), "p[%d]" % k, dev)
    for k, t in enumerate(u):
        _need(t, (H,), "u[%d]" % k, dev)
    _need(h, (B, L, H), "h", dev)
    _need(grad_h, (B, L, H), "grad_h", dev)
    if h0 is not None:
        _need(h0, (B, H), "h0", dev)
    if cell == CELL_LSTM:
        _need(c, (B, L, H), "c", dev)
        if c0 is not None:
            _need(c0, (B, H), "c0", dev)
        if grad_c is not None:
            _need(grad_c, (B, L, H), "grad_c", dev)
    gp = [torch.empty_like(h) for _ in range(ng)]
    gu = [torch.empty(H, dtype=torch.float32, device=dev) for _ in range(ng)] if want_u else None
    gh0 = torch.empty(B, H, dtype=torch.float32, device=dev) if want_h0 else None
    gc0 = torch.empty(B, H, dtype=torch.float32, device=dev) if (want_c0 and cell == CELL_LSTM) else None
    op = OP_GRU_ADJOINT if cell == CELL_GRU else OP_LSTM_ADJOINT
    ws, n = _workspace(op, B, L, H, dev, ws=ws)
    P = (ctypes.c_void_p * ng)(*[t.data_ptr() for t in p])
    U = (ctypes.c_void_p * ng)(*[t.data_ptr() for t in u])
    GP = (ctypes.c_void_p * ng)(*[t.data_ptr() for t in gp])
    GU = (ctypes.c_void_p * ng)(*[t.data_ptr() for t in gu]) if gu is not None else None
    _check(lib.pararnn_adjoint_backward(cell, B, L, H, P, U, _ptr(h0), _ptr(c0), _ptr(h), _ptr(c),
                                        _ptr(grad_h), _ptr(grad_c), GP, GU, _ptr(gh0), _ptr(gc0),
                                        _ptr(ws), n, _stream(dev)), "pararnn_adjoint_backward")
    return {"p": gp, "u": gu, "h0": gh0, "c0": gc0}


# ---------------------------------------------------------------- operators around the recurrences
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}   # PARARNN_F32, PARARNN_BF16
MAX_HEAD_DIM = 256


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _type_code(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be on a HIP device" % name)
    return code


def _need_typed(t, shape, dtype, name, device):
    """A dense tensor of the given shape, type and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


@functools.lru_cache(maxsize=1024)
def _linattn_ws(backward: int, *sizes) -> int:
    """pararnn_linattn_workspace_bytes, which depends on the sizes alone (asked once per set of sizes)."""
    return load_library().pararnn_linattn_workspace_bytes(backward, *sizes)


@functools.lru_cache(maxsize=1024)
def _layernorm_ws(rows: int, D: int) -> int:
    """pararnn_layernorm_workspace_bytes, likewise."""
    return load_library().pararnn_layernorm_workspace_bytes(rows, D)


def _linattn_views(tensors, shapes, names, dtype, device):
    """Checks the operands; the strides array the library takes, or None if all are dense."""
    dense = True
    for t, shape, name in zip(tensors, shapes, names):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if t.dtype != dtype or t.device != device or t.shape != shape:
            if t.dtype != dtype:
                raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
            if t.device != device:
                raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        if not t.is_contiguous():
            dense = False
            if t.shape[-1] > 1 and t.stride(-1) != 1:
                raise ValueError("the last dimension of %s must be dense" % name)
    if dense:
        return None
    st = []
    for t in tensors:
        s = t.stride()
        st += (s[0], s[1], s[2]) if t.dim() == 4 else (s[0], 0, s[1])
    return (ctypes.c_int64 * len(st))(*st)


def _linattn_check(q, v, seq: bool):
    code = _type_code(q, "q")
    shape = q.shape
    if len(shape) != 3 + seq or not isinstance(v, torch.Tensor) or v.dim() != 3 + seq:
        raise ValueError("q, k and v must be %s" % ("[B, L, H, d]" if seq else "[B, H, d]"))
    dk, dv = shape[-1], v.shape[-1]
    if 0 in shape or dv == 0:
        raise PararnnError("invalid sizes q %s, v %s" % (tuple(shape), tuple(v.shape)))
    if dk > MAX_HEAD_DIM or dv > MAX_HEAD_DIM:
        raise PararnnError("linear attention supports head sizes up to %d, got dk=%d dv=%d" % (MAX_HEAD_DIM, dk, dv))
    return code, dk, dv, shape


def linattn_forward(q, k, v, log_decay, state=None, *, scale=None, want_state=True, out=None, out_state=None,
                    ws=None):
    """Linear attention with a decay per head over whole sequences:
    S_t = e^g S_{t-1} + k_t^T v_t, o_t = scale q_t S_t, g = log_decay[head].

    q, k [B, L, H, dk], v [B, L, H, dv], fp32 or bf16, any strides with a dense
    last dimension; log_decay [H] fp32; state [B, H, dk, dv] fp32 or None.
    scale defaults to dk^-0.5.  Returns (o [B, L, H, dv], final state or None
    unless want_state).  out_state may be `state` itself.  bf16 outputs carry one
    or two roundings to bf16 on the way beside their own; states are fp32
    throughout.  The last bits of a row may differ in a batch of another size."""
    lib = load_library()
    code, dk, dv, kshape = _linattn_check(q, v, True)
    B, L, H, _ = kshape
    dev = q.device
    vshape, sshape = (B, L, H, dv), (B, H, dk, dv)
    st = _linattn_views((q, k, v), (kshape, kshape, vshape), ("q", "k", "v"), q.dtype, dev)
    _need_typed(log_decay, (H,), torch.float32, "log_decay", dev)
    if state is not None:
        _need_typed(state, sshape, torch.float32, "state", dev)
    if out is None:
        out = v.new_empty(vshape)
    else:
        _need_typed(out, vshape, q.dtype, "out", dev)
    if out_state is not None:
        _need_typed(out_state, sshape, torch.float32, "out_state", dev)
    elif want_state:
        out_state = log_decay.new_empty(sshape)
    buf, n = _workspace_of(_linattn_ws(0, code, B, L, H, dk, dv), dev, ws, True)
    _check(lib.pararnn_linattn_forward(code, B, L, H, dk, dv, _at(q), _at(k), _at(v), st, _at(log_decay),
                                       _at(state), dk ** -0.5 if scale is None else scale, _at(out),
                                       _at(out_state), _at(buf), n, _raw_stream(dev)), "pararnn_linattn_forward")
    return out, out_state


def linattn_backward(q, k, v, log_decay, grad_o, state=None, grad_state=None, *, scale=None, want_state=None,
                     ws=None):
    """Gradients of linattn_forward for dLoss/do = grad_o and dLoss/d(final
    state) = grad_state (None: zeros).  Returns (dq, dk, dv, dstate), dstate
    None unless want_state (default: whether a state is given).  log_decay is
    a constant of the model and gets no gradient."""
    lib = load_library()
    code, dk, dv, kshape = _linattn_check(q, v, True)
    B, L, H, _ = kshape
    dev = q.device
    vshape, sshape = (B, L, H, dv), (B, H, dk, dv)
    st = _linattn_views((q, k, v, grad_o), (kshape, kshape, vshape, vshape), ("q", "k", "v", "grad_o"), q.dtype, dev)
    _need_typed(log_decay, (H,), torch.float32, "log_decay", dev)
    for t, name in ((state, "state"), (grad_state, "grad_state")):
        if t is not None:
            _need_typed(t, sshape, torch.float32, name, dev)
    if want_state is None:
        want_state = state is not None
    gq, gk, gv = (torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v))
    gs = torch.empty(sshape, dtype=torch.float32, device=dev) if want_state else None
    buf, n = _workspace_of(_linattn_ws(1, code, B, L, H, dk, dv), dev, ws, True)
    _check(lib.pararnn_linattn_backward(code, B, L, H, dk, dv, _at(q), _at(k), _at(v), _at(grad_o), st,
                                        _at(log_decay), _at(state), _at(grad_state),
                                        dk ** -0.5 if scale is None else scale, _at(gq), _at(gk), _at(gv),
                                        _at(gs), _at(buf), n, _raw_stream(dev)), "pararnn_linattn_backward")
    return gq, gk, gv, gs


def linattn_step(q, k, v, log_decay, state, *, scale=None, out=None, out_state=None):
    """One token of linattn_forward (decoding): q, k [B, H, dk], v [B, H, dv],
    state [B, H, dk, dv].  Returns (o [B, H, dv], new state); out_state may be
    `state` itself."""
    lib = load_library()
    code, dk, dv, kshape = _linattn_check(q, v, False)
    B, H, _ = kshape
    dev = q.device
    vshape, sshape = (B, H, dv), (B, H, dk, dv)
    st = _linattn_views((q, k, v), (kshape, kshape, vshape), ("q", "k", "v"), q.dtype, dev)
    _need_typed(log_decay, (H,), torch.float32, "log_decay", dev)
    _need_typed(state, sshape, torch.float32, "state", dev)
    if out is None:
        out = v.new_empty(vshape)
    else:
        _need_typed(out, vshape, q.dtype, "out", dev)
    if out_state is None:
        out_state = log_decay.new_empty(sshape)
    else:
        _need_typed(out_state, sshape, torch.float32, "out_state", dev)
    _check(lib.pararnn_linattn_step(code, B, H, dk, dv, _at(q), _at(k), _at(v), st, _at(log_decay), _at(state),
                                    dk ** -0.5 if scale is None else scale, _at(out), _at(out_state),
                                    _raw_stream(dev)), "pararnn_linattn_step")
    return out, out_state


def _rows(x, name):
    """(rows, D) of a tensor normalised over its last dimension."""
    D = x.shape[-1] if x.dim() else 0
    if x.numel() == 0:
        raise PararnnError("%s is empty: %s" % (name, tuple(x.shape)))
    return x.numel() // D, D


def layernorm_forward(x, weight=None, bias=None, residual=None, *, eps=1e-5, out=None, out_sum=None):
    """Layer norm over the last dimension, after an optional residual sum:
    s = x + residual (in x's type), y = (s - mean) rstd weight + bias.

    x, residual [..., D] fp32 or bf16; weight, bias [D] fp32 or None.  Returns
    (y, s, mean, rstd): s is x itself without a residual, mean and rstd [...]
    fp32 are what layernorm_backward takes."""
    lib = load_library()
    code = _type_code(x, "x")
    rows, D = _rows(x, "x")
    dev, shape = x.device, x.shape
    _need_typed(x, shape, x.dtype, "x", dev)
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _need_typed(t, (D,), torch.float32, name, dev)
    y = torch.empty_like(x) if out is None else out
    if out is not None:
        _need_typed(out, shape, x.dtype, "out", dev)
    s = None
    if residual is not None:
        _need_typed(residual, shape, x.dtype, "residual", dev)
        s = torch.empty_like(x) if out_sum is None else out_sum
        _need_typed(s, shape, x.dtype, "out_sum", dev)
    elif out_sum is not None:
        raise ValueError("out_sum is given without a residual")
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    _check(lib.pararnn_layernorm_forward(code, rows, D, _at(x), _at(residual), _at(weight), _at(bias), eps,
                                         _at(s), _at(y), _at(mean), _at(rstd), _raw_stream(dev)),
           "pararnn_layernorm_forward")
    return y, x if s is None else s, mean, rstd


def layernorm_backward(s, weight, mean, rstd, grad_y, grad_sum=None, *, want_w=True, want_b=True, ws=None):
    """Gradients of layernorm_forward: s, mean, rstd are its results, grad_sum
    (None: zero) what reaches the sum past the norm.  Returns (dx, dweight,
    dbias); dx is the gradient of x and of the residual alike."""
    lib = load_library()
    code = _type_code(s, "s")
    rows, D = _rows(s, "s")
    dev, shape = s.device, s.shape
    _need_typed(s, shape, s.dtype, "s", dev)
    _need_typed(grad_y, shape, s.dtype, "grad_y", dev)
    if grad_sum is not None:
        _need_typed(grad_sum, shape, s.dtype, "grad_sum", dev)
    if weight is not None:
        _need_typed(weight, (D,), torch.float32, "weight", dev)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _need_typed(t, shape[:-1], torch.float32, name, dev)
    dx = torch.empty_like(s)
    gw = torch.empty(D, dtype=torch.float32, device=dev) if want_w else None
    gb = torch.empty(D, dtype=torch.float32, device=dev) if want_b else None
    buf, n = _workspace_of(_layernorm_ws(rows, D), dev, ws, True) if want_w or want_b else (None, 0)
    _check(lib.pararnn_layernorm_backward(code, rows, D, _at(s), _at(weight), _at(mean), _at(rstd), _at(grad_y),
                                          _at(grad_sum), _at(dx), _at(gw), _at(gb), _at(buf), n, _raw_stream(dev)),
           "pararnn_layernorm_backward")
    return dx, gw, gb


def _ids(ids, device):
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    if ids.device != device:
        raise ValueError("ids is on %s, expected %s" % (ids.device, device))
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    if ids.numel() == 0:
        raise PararnnError("ids is empty")
    return ids.numel(), ids.element_size()


def embedding_forward(ids, table, *, scale=1.0, out=None):
    """scale * table[ids]: ids [...] int32 or int64, table [V, D] fp32 or bf16;
    returns [..., D].  An id outside [0, V) gives a row of NaN."""
    lib = load_library()
    code = _type_code(table, "table")
    dev = table.device
    if table.dim() != 2 or table.numel() == 0:
        raise ValueError("table must be [V, D], got %s" % (tuple(table.shape),))
    V, D = table.shape
    _need_typed(table, (V, D), table.dtype, "table", dev)
    N, nb = _ids(ids, dev)
    if out is None:
        out = torch.empty((*ids.shape, D), dtype=table.dtype, device=dev)
    else:
        _need_typed(out, (*ids.shape, D), table.dtype, "out", dev)
    _check(lib.pararnn_embedding_forward(code, N, V, D, _at(ids), nb, _at(table), scale, _at(out), _raw_stream(dev)),
           "pararnn_embedding_forward")
    return out


def embedding_backward(ids, grad, num_rows, *, scale=1.0, padding_idx=None, out=None, ws=None):
    """Gradient of embedding_forward's table: [num_rows, D] in grad's type,
    row r = scale * the sum of grad over the positions where ids is r (in
    their order), zeros elsewhere and at padding_idx."""
    lib = load_library()
    code = _type_code(grad, "grad")
    dev = grad.device
    N, nb = _ids(ids, dev)
    if grad.dim() < 1 or grad.shape[-1] == 0:
        raise ValueError("grad must be [..., D]")
    D, V = grad.shape[-1], int(num_rows)
    _need_typed(grad, (*ids.shape, D), grad.dtype, "grad", dev)
    if V < 1:
        raise PararnnError("num_rows must be positive, got %d" % V)
    if padding_idx is not None and not 0 <= padding_idx < V:
        raise ValueError("padding_idx must be in [0, %d), got %s" % (V, padding_idx))
    if out is None:
        out = torch.empty((V, D), dtype=grad.dtype, device=dev)
    else:
        _need_typed(out, (V, D), grad.dtype, "out", dev)
    n = lib.pararnn_embedding_workspace_bytes(N, V, D)
    if n == 0:
        raise PararnnError("invalid sizes N=%d V=%d D=%d" % (N, V, D))
    buf, n = _workspace_of(n, dev, ws, True)
    _check(lib.pararnn_embedding_backward(code, N, V, D, _at(ids), nb, _at(grad), scale,
                                          -1 if padding_idx is None else padding_idx, _at(out), _at(buf), n,
                                          _raw_stream(dev)), "pararnn_embedding_backward")
    return out
