"""Thin Python binding of libint4vh.so (the C ABI declared in include/int4vh.h).

Argument marshalling only: every step of the verify path runs in the HIP
kernels of the library.  torch tensors supply device memory and the current
stream; outputs are allocated with torch on the input's device.  If the
library has not been built the first call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libint4vh.so")

OK, EINVAL, EALIGN, EWORKSPACE, EHIP, EUNSUPPORTED, ESCRATCH = 0, -1, -2, -3, -4, -5, -6

_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load (once) and return the library; raise if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(path)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.verify_lm_head_int4_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.verify_lm_head_int4_workspace_bytes.restype = sz
        L.verify_lm_head_int4_sampled_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.verify_lm_head_int4_sampled_workspace_bytes.restype = sz
        L.verify_lm_head_int4_workspace_init.argtypes = [P, sz, P]
        L.verify_lm_head_int4_workspace_init.restype = i32
        L.verify_lm_head_int4.argtypes = [P, P, P, P, i32, i32, i32, P, P, P, P, P, sz, P]
        L.verify_lm_head_int4.restype = i32
        L.verify_lm_head_int4_batch.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P, P, P, P,
                                                sz, P]
        L.verify_lm_head_int4_batch.restype = i32
        L.verify_lm_head_int4_batch_timed.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P, P, P,
                                                      P, sz, P, P, P]
        L.verify_lm_head_int4_batch_timed.restype = i32
        L.verify_lm_head_int4_batch_noalloc.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P, P, P,
                                                        P]
        L.verify_lm_head_int4_batch_noalloc.restype = i32
        L.verify_lm_head_int4_check_weights.argtypes = [P, i32, i32, P, P]
        L.verify_lm_head_int4_check_weights.restype = i32
        L.verify_lm_head_int4_status_string.argtypes = [i32]
        L.verify_lm_head_int4_status_string.restype = ctypes.c_char_p
        L.verify_lm_head_int4_last_error.argtypes = []
        L.verify_lm_head_int4_last_error.restype = ctypes.c_char_p
        L.verify_lm_head_int4_mapped.argtypes = [P, P, P, P, P, i32, i32, i32, i32, P, P, P, P,
                                                 P, sz, P]
        L.verify_lm_head_int4_mapped.restype = i32
        L.verify_lm_head_int4_check_vocab_map.argtypes = [P, i32, P, P]
        L.verify_lm_head_int4_check_vocab_map.restype = i32
        L.verify_lm_head_int4_sampled.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                                  ctypes.c_float, P, P, P, P, P, P, P, P, sz, P]
        L.verify_lm_head_int4_sampled.restype = i32
        L.verify_lm_head_int4_sampled_timed.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                                        ctypes.c_float, P, P, P, P, P, P, P, P, sz,
                                                        P, P, P]
        L.verify_lm_head_int4_sampled_timed.restype = i32
        # read-only streaming reference (include/int4vh_probe.h)
        L.int4vh_stream_read.argtypes = [P, sz, i32, P, P, P, P]
        L.int4vh_stream_read.restype = i32
        # context-copy drafter (include/int4vh_drafter.h)
        L.context_copy_propose.argtypes = [P, P, i32, P, i32, i32, i32, P, P, P, P, P]
        L.context_copy_propose.restype = i32
        L.context_copy_propose_timed.argtypes = [P, P, i32, P, i32, i32, i32, P, P, P, P, P, P, P]
        L.context_copy_propose_timed.restype = i32
        # offline requantisation (include/int4vh_requant.h)
        L.requant_lm_head_int4_amax.argtypes = [P, i32, i32, i32, P, i32, P]
        L.requant_lm_head_int4_amax.restype = i32
        L.requant_lm_head_int4_scales.argtypes = [P, i32, P, P]
        L.requant_lm_head_int4_scales.restype = i32
        L.requant_lm_head_int4_pack.argtypes = [P, i32, i32, i32, P, P, P]
        L.requant_lm_head_int4_pack.restype = i32
        L.requant_lm_head_int4_pack_timed.argtypes = [P, i32, i32, i32, P, P, P, P, P]
        L.requant_lm_head_int4_pack_timed.restype = i32
        L.requant_lm_head_int4.argtypes = [P, i32, i32, i32, P, i32, i32, P, P, P, P]
        L.requant_lm_head_int4.restype = i32
        # row operators in front of the products (include/int4vh_norm.h)
        i64, f32 = ctypes.c_int64, ctypes.c_float
        L.rms_norm_rows.argtypes = [P, i64, P, i64, i32, P, i32, i32, i32, f32, P, P, i32, P]
        L.rms_norm_rows.restype = i32
        L.rms_norm_rows_int8.argtypes = [P, i64, P, i64, i32, P, i32, P, i32, i32, f32, P, P, P, P]
        L.rms_norm_rows_int8.restype = i32
        L.quantize_rows_int8.argtypes = [P, i64, i32, P, i32, i32, P, P, P]
        L.quantize_rows_int8.restype = i32
        L.rms_norm_block_rows.argtypes = [P, i64, P, i64, P, i64, i32, i32, P, P, i32, f32, i32, i32, f32, P, P, i32,
                                          P]
        L.rms_norm_block_rows.restype = i32
        L.rms_norm_block_rows_int8.argtypes = [P, i64, P, i64, P, i64, i32, i32, P, P, i32, P, f32, i32, i32, f32, P,
                                               P, P, P]
        L.rms_norm_block_rows_int8.restype = i32
        # linear layers on packed int4 weights (include/int4vh_linear.h)
        L.linear_int4_rows_workspace_bytes.argtypes = [i32, i32, i32]
        L.linear_int4_rows_workspace_bytes.restype = sz
        L.linear_int4_rows.argtypes = [P, i64, P, P, P, P, i32, P, i64, i32, i32, i32, P, i64, i32, P, sz, P]
        L.linear_int4_rows.restype = i32
        # 4-bit floating point (include/int4vh_mxfp4.h)
        L.quantize_rows_mxfp4.argtypes = [P, i64, i32, i32, i32, P, P, P]
        L.quantize_rows_mxfp4.restype = i32
        L.dequantize_rows_mxfp4.argtypes = [P, P, i32, i32, P, i32, P]
        L.dequantize_rows_mxfp4.restype = i32
        L.linear_mxfp4_rows_workspace_bytes.argtypes = [i32, i32, i32]
        L.linear_mxfp4_rows_workspace_bytes.restype = sz
        L.linear_mxfp4_rows.argtypes = [P, P, P, P, P, i32, P, i64, i32, i32, i32, P, i64, i32, P, sz, P]
        L.linear_mxfp4_rows.restype = i32
        # rules on logits (include/int4vh_logits.h)
        L.logit_rules_apply.argtypes = [P, i64, i32, P, i32, i32, i32, P, P, i64, P]
        L.logit_rules_apply.restype = i32
        L.logit_rules_verify_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.logit_rules_verify_workspace_bytes.restype = sz
        L.logit_rules_verify.argtypes = [P, i64, i32, P, P, P, i32, i32, i32, P, i32, f32, P, P, P, P, P, P, P,
                                         P, sz, P]
        L.logit_rules_verify.restype = i32
        L.verify_lm_head_int4_ruled_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.verify_lm_head_int4_ruled_workspace_bytes.restype = sz
        L.verify_lm_head_int4_ruled.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, P, i32, f32, P, P, P, P, P,
                                                P, P, P, sz, P]
        L.verify_lm_head_int4_ruled.restype = i32
        # tokens drawn from logits (include/int4vh_sample.h)
        L.sample_logits_workspace_bytes.argtypes = [i32, i32, i32]
        L.sample_logits_workspace_bytes.restype = sz
        L.sample_logits_rows.argtypes = [P, i64, i32, P, i32, i32, i32, P, P, P, P, P, P, P, P, P, sz, P]
        L.sample_logits_rows.restype = i32
        _lib = L
        return L


def _raise(status: int, what: str):
    L = load_library()
    msg = L.verify_lm_head_int4_status_string(status).decode()
    if status == EHIP:
        msg += ": " + L.verify_lm_head_int4_last_error().decode()
        # a workspace has to be initialised again after such an error
        _ws_cache.clear()
    raise RuntimeError(f"{what}: {msg} (status {status})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def workspace_bytes(R: int, T: int, V: int, H: int) -> int:
    return int(load_library().verify_lm_head_int4_workspace_bytes(R, T, V, H))


def sampled_workspace_bytes(R: int, T: int, V: int, H: int) -> int:
    return int(load_library().verify_lm_head_int4_sampled_workspace_bytes(R, T, V, H))


class Workspace:
    """A device workspace for verify calls, initialised on creation.  Calls
    that share a Workspace must not be in flight at the same time, replays of
    graphs that were captured with it among them; a graph does not keep it
    alive.  Calls without one use one per stream, or under torch's capture one
    per call, which is part of the graph's memory."""

    def __init__(self, nbytes: int, device):
        self.nbytes = int(nbytes)
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        st = load_library().verify_lm_head_int4_workspace_init(
            _ptr(self.tensor), self.nbytes, _stream_ptr(self.tensor.device))
        if st != OK:
            _raise(st, "workspace_init")


_ws_cache: dict = {}


def _default_workspace(device, nbytes: int) -> Workspace:
    # A graph keeps the addresses it was captured with, while an eager call may
    # replace the stream's workspace by a larger one, and a replay may run
    # beside the stream's eager calls: a call under capture gets its own, from
    # the graph's memory, which the graph initialises itself.
    if _on(device.index, torch.cuda.is_current_stream_capturing):
        return Workspace(nbytes, device)
    # one per (device, current stream): calls on one stream are ordered
    key = (device.index, _raw_stream(device.index))
    ws = _ws_cache.get(key)
    if ws is None or ws.nbytes < nbytes:
        ws = Workspace(nbytes, device)
        _ws_cache[key] = ws
    return ws


def _check(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _event_handle(ev, stream):
    """Raw hipEvent_t of a torch.cuda.Event (created by a first record);
    None gives a null handle (that end of the kernel is not timed)."""
    if ev is None:
        return ctypes.c_void_p(None)
    if ev.cuda_event == 0:
        ev.record(stream)
    return ctypes.c_void_p(ev.cuda_event)


def verify_batch(hidden, packed_w, scales, draft_ids=None, *, R: int | None = None,
                 logits: bool = False, workspace: Workspace | None = None, events=None):
    """R requests x T positions.  hidden: float16 [R, T, H] (or [R*T, H] with
    R given); packed_w: uint8 [V, H/2]; scales: float16 [H]; draft_ids: int32
    [R, T-1] (None when T == 1).  Returns (logits_max [R*T], argmax_ids [R*T],
    n_accepted [R]) and, with logits=True, logits [R*T, V] as a 4th item.
    events=(before, after), two torch.cuda.Event(enable_timing=True), take
    the start and end timestamps of the main verify kernel's own dispatch
    (the instrumented entry point verify_lm_head_int4_batch_timed; not for
    use under graph capture)."""
    if hidden.dim() == 3:
        R, T, H = hidden.shape
        hidden = hidden.reshape(R * T, H)
    else:
        if R is None:
            raise ValueError("R is required for a 2-D hidden tensor")
        T = hidden.shape[0] // R
        H = hidden.shape[1]
    _check(hidden, "hidden", torch.float16, 2)
    _check(packed_w, "packed_w", torch.uint8, 2)
    _check(scales, "scales", torch.float16, 1)
    V = packed_w.shape[0]
    if packed_w.shape[1] * 2 != H or scales.shape[0] != H or hidden.shape[0] != R * T:
        raise ValueError("shape mismatch between hidden, packed_w and scales")
    dev = hidden.device
    if T > 1:
        if draft_ids is None:
            raise ValueError("draft_ids is required when T > 1")
        _check(draft_ids, "draft_ids", torch.int32)
        if draft_ids.numel() != R * (T - 1):
            raise ValueError("draft_ids must hold R*(T-1) ids")
    else:
        draft_ids = None
    M = R * T
    lmax = torch.empty(M, dtype=torch.float32, device=dev)
    amax = torch.empty(M, dtype=torch.int32, device=dev)
    nacc = torch.empty(R, dtype=torch.int32, device=dev)
    lout = torch.empty((M, V), dtype=torch.float32, device=dev) if logits else None
    L = load_library()
    need = L.verify_lm_head_int4_workspace_bytes(R, T, V, H)
    if need == 0:
        _raise(EINVAL, "verify")
    ws = workspace if workspace is not None else _default_workspace(dev, need)
    args = (_ptr(hidden), _ptr(packed_w), _ptr(scales), _ptr(draft_ids), R, T, V, H, _ptr(lmax),
            _ptr(amax), _ptr(nacc), _ptr(lout), _ptr(ws.tensor), ws.nbytes, _stream_ptr(dev))
    if events is None:
        st = L.verify_lm_head_int4_batch(*args)
    else:
        stream = torch.cuda.current_stream(dev)
        st = L.verify_lm_head_int4_batch_timed(*args, _event_handle(events[0], stream),
                                               _event_handle(events[1], stream))
    if st != OK:
        _raise(st, "verify_lm_head_int4_batch")
    return (lmax, amax, nacc, lout) if logits else (lmax, amax, nacc)


def verify_batch_noalloc(hidden, packed_w, scales, draft_ids=None, *, R: int | None = None,
                         logits: bool = False, out=None):
    """verify_batch through the entry point that allocates nothing
    (verify_lm_head_int4_batch_noalloc: the library's static per-device
    scratch replaces the workspace).  out=(logits_max, argmax_ids,
    n_accepted[, logits]) supplies preallocated outputs (as a caller under
    graph capture would); otherwise they are allocated here, by torch.  Calls
    that overlap in time on one device race on the shared scratch."""
    if hidden.dim() == 3:
        R, T, H = hidden.shape
        hidden = hidden.reshape(R * T, H)
    else:
        if R is None:
            raise ValueError("R is required for a 2-D hidden tensor")
        T = hidden.shape[0] // R
        H = hidden.shape[1]
    _check(hidden, "hidden", torch.float16, 2)
    _check(packed_w, "packed_w", torch.uint8, 2)
    _check(scales, "scales", torch.float16, 1)
    V = packed_w.shape[0]
    if packed_w.shape[1] * 2 != H or scales.shape[0] != H or hidden.shape[0] != R * T:
        raise ValueError("shape mismatch between hidden, packed_w and scales")
    dev = hidden.device
    if T > 1:
        if draft_ids is None:
            raise ValueError("draft_ids is required when T > 1")
        _check(draft_ids, "draft_ids", torch.int32)
        if draft_ids.numel() != R * (T - 1):
            raise ValueError("draft_ids must hold R*(T-1) ids")
    else:
        draft_ids = None
    M = R * T
    if out is not None:
        lmax, amax, nacc = out[0], out[1], out[2]
        lout = out[3] if len(out) > 3 else None
        _check(lmax, "logits_max", torch.float32)
        _check(amax, "argmax_ids", torch.int32)
        _check(nacc, "n_accepted", torch.int32)
        if lmax.numel() != M or amax.numel() != M or nacc.numel() != R:
            raise ValueError("output sizes do not match R*T rows and R requests")
        if lout is not None:
            _check(lout, "logits", torch.float32)
            if lout.numel() != M * V:
                raise ValueError("logits must hold R*T*V values")
    else:
        lmax = torch.empty(M, dtype=torch.float32, device=dev)
        amax = torch.empty(M, dtype=torch.int32, device=dev)
        nacc = torch.empty(R, dtype=torch.int32, device=dev)
        lout = torch.empty((M, V), dtype=torch.float32, device=dev) if logits else None
    st = load_library().verify_lm_head_int4_batch_noalloc(
        _ptr(hidden), _ptr(packed_w), _ptr(scales), _ptr(draft_ids), R, T, V, H, _ptr(lmax),
        _ptr(amax), _ptr(nacc), _ptr(lout), _stream_ptr(dev))
    if st != OK:
        _raise(st, "verify_batch_noalloc")
    return (lmax, amax, nacc, lout) if lout is not None else (lmax, amax, nacc)


def verify_mapped(hidden, packed_w, scales, vocab_ids, draft_ids=None, *, R: int | None = None,
                  logits: bool = False, workspace: Workspace | None = None):
    """Verify through a head whose rows are a subset of the vocabulary:
    vocab_ids (int32 [V], strictly increasing) maps each head row to its
    token id; argmax_ids are token ids and draft_ids are compared with them.
    Otherwise as verify_batch (hidden [R, T, H], or [R*T, H] with R)."""
    if hidden.dim() == 3:
        R, T, H = hidden.shape
        hidden = hidden.reshape(R * T, H)
    else:
        if R is None:
            raise ValueError("R is required for a 2-D hidden tensor")
        T = hidden.shape[0] // R
        H = hidden.shape[1]
    _check(hidden, "hidden", torch.float16, 2)
    _check(packed_w, "packed_w", torch.uint8, 2)
    _check(scales, "scales", torch.float16, 1)
    _check(vocab_ids, "vocab_ids", torch.int32, 1)
    V = packed_w.shape[0]
    if packed_w.shape[1] * 2 != H or scales.shape[0] != H or hidden.shape[0] != R * T:
        raise ValueError("shape mismatch between hidden, packed_w and scales")
    if vocab_ids.shape[0] != V:
        raise ValueError("vocab_ids must hold one id per head row")
    dev = hidden.device
    if T > 1:
        if draft_ids is None:
            raise ValueError("draft_ids is required when T > 1")
        _check(draft_ids, "draft_ids", torch.int32)
        if draft_ids.numel() != R * (T - 1):
            raise ValueError("draft_ids must hold R*(T-1) ids")
    else:
        draft_ids = None
    M = R * T
    lmax = torch.empty(M, dtype=torch.float32, device=dev)
    amax = torch.empty(M, dtype=torch.int32, device=dev)
    nacc = torch.empty(R, dtype=torch.int32, device=dev)
    lout = torch.empty((M, V), dtype=torch.float32, device=dev) if logits else None
    L = load_library()
    need = L.verify_lm_head_int4_workspace_bytes(R, T, V, H)
    if need == 0:
        _raise(EINVAL, "verify_mapped")
    ws = workspace if workspace is not None else _default_workspace(dev, need)
    st = L.verify_lm_head_int4_mapped(_ptr(hidden), _ptr(packed_w), _ptr(scales), _ptr(vocab_ids),
                                      _ptr(draft_ids), R, T, V, H, _ptr(lmax), _ptr(amax), _ptr(nacc),
                                      _ptr(lout), _ptr(ws.tensor), ws.nbytes, _stream_ptr(dev))
    if st != OK:
        _raise(st, "verify_lm_head_int4_mapped")
    return (lmax, amax, nacc, lout) if logits else (lmax, amax, nacc)


def verify_sampled(hidden, packed_w, scales, draft_ids=None, draft_probs=None, uniforms=None, *,
                   top_k: int, temperature: float = 1.0, R: int | None = None,
                   workspace: Workspace | None = None, events=None, want_lse: bool = False):
    """Sampled verification for R*T <= 4096 rows: top-k sampling at a
    temperature (top_k >= 1) or sampling over the whole vocabulary
    (top_k == 0).  hidden: float16 [R, T, H] (or [R*T, H] with R); draft_ids
    int32, draft_probs and uniforms float32, each [R, T-1] (None when T == 1).
    Returns (logits_max [R*T], argmax_ids [R*T], topk_ids [R*T, k],
    topk_logits [R*T, k], p_draft [R, T-1], n_accepted [R], lse [R*T]) (the
    top-k outputs are None when top_k == 0; lse, the log-sum-exp of
    logit / temperature over the vocabulary, is None unless want_lse or
    top_k == 0).  events=(before, after) take the start and end timestamps of
    the main verify kernel's dispatch.  Above 64 rows the workspace also
    holds the call's logits (sampled_workspace_bytes)."""
    if hidden.dim() == 3:
        R, T, H = hidden.shape
        hidden = hidden.reshape(R * T, H)
    else:
        if R is None:
            raise ValueError("R is required for a 2-D hidden tensor")
        T = hidden.shape[0] // R
        H = hidden.shape[1]
    _check(hidden, "hidden", torch.float16, 2)
    _check(packed_w, "packed_w", torch.uint8, 2)
    _check(scales, "scales", torch.float16, 1)
    V = packed_w.shape[0]
    if packed_w.shape[1] * 2 != H or scales.shape[0] != H or hidden.shape[0] != R * T:
        raise ValueError("shape mismatch between hidden, packed_w and scales")
    dev = hidden.device
    if T > 1:
        for t, n, dt in ((draft_ids, "draft_ids", torch.int32), (draft_probs, "draft_probs", torch.float32),
                         (uniforms, "uniforms", torch.float32)):
            if t is None:
                raise ValueError(f"{n} is required when T > 1")
            _check(t, n, dt)
            if t.numel() != R * (T - 1):
                raise ValueError(f"{n} must hold R*(T-1) values")
    else:
        draft_ids = draft_probs = uniforms = None
    M = R * T
    k = int(top_k)
    lmax = torch.empty(M, dtype=torch.float32, device=dev)
    amax = torch.empty(M, dtype=torch.int32, device=dev)
    tids = torch.empty((M, k), dtype=torch.int32, device=dev) if k > 0 else None
    tlog = torch.empty((M, k), dtype=torch.float32, device=dev) if k > 0 else None
    lse = torch.empty(M, dtype=torch.float32, device=dev) if (want_lse or k == 0) else None
    pdr = torch.empty((R, max(T - 1, 1)), dtype=torch.float32, device=dev)
    nacc = torch.empty(R, dtype=torch.int32, device=dev)
    L = load_library()
    need = L.verify_lm_head_int4_sampled_workspace_bytes(R, T, V, H)
    if need == 0:
        _raise(EINVAL, "verify_sampled")
    ws = workspace if workspace is not None else _default_workspace(dev, need)
    args = (_ptr(hidden), _ptr(packed_w), _ptr(scales), _ptr(draft_ids), _ptr(draft_probs),
            _ptr(uniforms), R, T, V, H, k, float(temperature), _ptr(lmax), _ptr(amax), _ptr(tids),
            _ptr(tlog), _ptr(lse), _ptr(pdr), _ptr(nacc), _ptr(ws.tensor), ws.nbytes, _stream_ptr(dev))
    if events is None:
        st = L.verify_lm_head_int4_sampled(*args)
    else:
        stream = torch.cuda.current_stream(dev)
        st = L.verify_lm_head_int4_sampled_timed(*args, _event_handle(events[0], stream),
                                                 _event_handle(events[1], stream))
    if st != OK:
        _raise(st, "verify_lm_head_int4_sampled")
    return lmax, amax, tids, tlog, pdr[:, : max(T - 1, 0)], nacc, lse


def check_vocab_map(vocab_ids) -> torch.Tensor:
    """Number of positions where vocab_ids is not strictly increasing and
    non-negative, as an int32 [1] device tensor (asynchronous)."""
    _check(vocab_ids, "vocab_ids", torch.int32, 1)
    out = torch.empty(1, dtype=torch.int32, device=vocab_ids.device)
    st = load_library().verify_lm_head_int4_check_vocab_map(
        _ptr(vocab_ids), vocab_ids.shape[0], _ptr(out), _stream_ptr(vocab_ids.device))
    if st != OK:
        _raise(st, "check_vocab_map")
    return out


def verify(hidden, packed_w, scales, draft_ids=None, *, logits: bool = False,
           workspace: Workspace | None = None):
    """One request.  hidden: float16 [T, H]; draft_ids: int32 [T-1] or None
    when T == 1.  Returns (logits_max [T], argmax_ids [T], n_accepted [1])
    and logits [T, V] with logits=True."""
    _check(hidden, "hidden", torch.float16, 2)
    _check(packed_w, "packed_w", torch.uint8, 2)
    _check(scales, "scales", torch.float16, 1)
    T, H = hidden.shape
    V = packed_w.shape[0]
    if packed_w.shape[1] * 2 != H or scales.shape[0] != H:
        raise ValueError("shape mismatch between hidden, packed_w and scales")
    dev = hidden.device
    if T > 1:
        if draft_ids is None:
            raise ValueError("draft_ids is required when T > 1")
        _check(draft_ids, "draft_ids", torch.int32)
        if draft_ids.numel() != T - 1:
            raise ValueError("draft_ids must hold T-1 ids")
    else:
        draft_ids = None
    lmax = torch.empty(T, dtype=torch.float32, device=dev)
    amax = torch.empty(T, dtype=torch.int32, device=dev)
    nacc = torch.empty(1, dtype=torch.int32, device=dev)
    lout = torch.empty((T, V), dtype=torch.float32, device=dev) if logits else None
    L = load_library()
    need = L.verify_lm_head_int4_workspace_bytes(1, T, V, H)
    if need == 0:
        _raise(EINVAL, "verify")
    ws = workspace if workspace is not None else _default_workspace(dev, need)
    st = L.verify_lm_head_int4(_ptr(hidden), _ptr(packed_w), _ptr(scales), _ptr(draft_ids),
                               T, V, H, _ptr(lmax), _ptr(amax), _ptr(nacc), _ptr(lout),
                               _ptr(ws.tensor), ws.nbytes, _stream_ptr(dev))
    if st != OK:
        _raise(st, "verify_lm_head_int4")
    return (lmax, amax, nacc, lout) if logits else (lmax, amax, nacc)


def check_weights(packed_w) -> torch.Tensor:
    """Number of illegal (0x8) nibbles of a packed head, as an int32 [1]
    device tensor (asynchronous)."""
    _check(packed_w, "packed_w", torch.uint8, 2)
    V, Hh = packed_w.shape
    out = torch.empty(1, dtype=torch.int32, device=packed_w.device)
    st = load_library().verify_lm_head_int4_check_weights(
        _ptr(packed_w), V, 2 * Hh, _ptr(out), _stream_ptr(packed_w.device))
    if st != OK:
        _raise(st, "check_weights")
    return out


# ---------------------------------------------------------------- requantisation

F16, BF16 = 0, 1
_DTYPES = {torch.float16: F16, torch.bfloat16: BF16}


def _dtype_code(t, name):
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return _DTYPES[t.dtype]


def requant_amax(acts, amax=None, *, accumulate: bool = False) -> torch.Tensor:
    """Per-channel max |acts| of calibration rows acts [N, H] (float16 or
    bfloat16) into amax (float32 [H]); with accumulate=True the running
    maximum of an existing amax.  Returns amax (asynchronous)."""
    if not isinstance(acts, torch.Tensor) or not acts.is_cuda:
        raise TypeError("acts must be a CUDA (HIP) tensor")
    dt = _dtype_code(acts, "acts")
    _check(acts, "acts", acts.dtype, 2)
    N, H = acts.shape
    if amax is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing amax")
        amax = torch.empty(H, dtype=torch.float32, device=acts.device)
    _check(amax, "amax", torch.float32, 1)
    if amax.shape[0] != H:
        raise ValueError("amax must hold H values")
    st = load_library().requant_lm_head_int4_amax(_ptr(acts), dt, N, H, _ptr(amax), int(accumulate),
                                                  _stream_ptr(acts.device))
    if st != OK:
        _raise(st, "requant_lm_head_int4_amax")
    return amax


def requant_scales(amax) -> torch.Tensor:
    """float16 scales [H] = amax / 7 (binary32 division, rounded to binary16)."""
    _check(amax, "amax", torch.float32, 1)
    H = amax.shape[0]
    scales = torch.empty(H, dtype=torch.float16, device=amax.device)
    st = load_library().requant_lm_head_int4_scales(_ptr(amax), H, _ptr(scales),
                                                    _stream_ptr(amax.device))
    if st != OK:
        _raise(st, "requant_lm_head_int4_scales")
    return scales


def requant_pack(W, scales, *, events=None) -> torch.Tensor:
    """Quantise the head W [V, H] (float16 or bfloat16) with per-channel
    scales (float16 [H]) and pack it: uint8 [V, H/2] in the verify layout.
    events=(before, after) take the start and end timestamps of the pack
    kernel's dispatch."""
    if not isinstance(W, torch.Tensor) or not W.is_cuda:
        raise TypeError("W must be a CUDA (HIP) tensor")
    dt = _dtype_code(W, "W")
    _check(W, "W", W.dtype, 2)
    _check(scales, "scales", torch.float16, 1)
    V, H = W.shape
    if scales.shape[0] != H:
        raise ValueError("scales must hold H values")
    packed = torch.empty((V, H // 2), dtype=torch.uint8, device=W.device)
    L = load_library()
    if events is None:
        st = L.requant_lm_head_int4_pack(_ptr(W), dt, V, H, _ptr(scales), _ptr(packed),
                                         _stream_ptr(W.device))
    else:
        stream = torch.cuda.current_stream(W.device)
        st = L.requant_lm_head_int4_pack_timed(_ptr(W), dt, V, H, _ptr(scales), _ptr(packed),
                                               _stream_ptr(W.device),
                                               _event_handle(events[0], stream),
                                               _event_handle(events[1], stream))
    if st != OK:
        _raise(st, "requant_lm_head_int4_pack")
    return packed


def requantize(W, acts):
    """The whole offline step for one calibration batch: returns (packed
    uint8 [V, H/2], scales float16 [H], amax float32 [H])."""
    for t, n in ((W, "W"), (acts, "acts")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{n} must be a CUDA (HIP) tensor")
    wdt, adt = _dtype_code(W, "W"), _dtype_code(acts, "acts")
    _check(W, "W", W.dtype, 2)
    _check(acts, "acts", acts.dtype, 2)
    V, H = W.shape
    N = acts.shape[0]
    if acts.shape[1] != H:
        raise ValueError("acts and W must have the same H")
    dev = W.device
    amax = torch.empty(H, dtype=torch.float32, device=dev)
    scales = torch.empty(H, dtype=torch.float16, device=dev)
    packed = torch.empty((V, H // 2), dtype=torch.uint8, device=dev)
    st = load_library().requant_lm_head_int4(_ptr(W), wdt, V, H, _ptr(acts), adt, N, _ptr(amax),
                                             _ptr(scales), _ptr(packed), _stream_ptr(dev))
    if st != OK:
        _raise(st, "requant_lm_head_int4")
    return packed, scales, amax


# ---------------------------------------------------------------- context-copy drafter

def context_copy(prompts, offsets, keys, *, n_min: int = 1, n_out: int = 8, events=None):
    """Propose the tokens copied from each request's prompt.  prompts: int32
    [total] (all prompts back to back); offsets: int64 [R+1]; keys: int32
    [R, n_max] (the last n_max tokens of each sequence).  Returns (tokens
    int32 [R, n_out] (-1 past count), count [R], match_end [R], match_len
    [R]).  events=(before, after) take the kernel's dispatch start and end."""
    _check(prompts, "prompts", torch.int32, 1)
    _check(offsets, "offsets", torch.int64, 1)
    _check(keys, "keys", torch.int32, 2)
    R, n_max = keys.shape
    if offsets.shape[0] != R + 1:
        raise ValueError("offsets must hold R+1 values")
    dev = prompts.device
    tok = torch.empty((R, n_out), dtype=torch.int32, device=dev)
    cnt = torch.empty(R, dtype=torch.int32, device=dev)
    end = torch.empty(R, dtype=torch.int32, device=dev)
    ln = torch.empty(R, dtype=torch.int32, device=dev)
    L = load_library()
    args = (_ptr(prompts), _ptr(offsets), R, _ptr(keys), n_max, n_min, n_out, _ptr(tok), _ptr(cnt),
            _ptr(end), _ptr(ln), _stream_ptr(dev))
    if events is None:
        st = L.context_copy_propose(*args)
    else:
        stream = torch.cuda.current_stream(dev)
        st = L.context_copy_propose_timed(*args, _event_handle(events[0], stream),
                                          _event_handle(events[1], stream))
    if st != OK:
        _raise(st, "context_copy_propose")
    return tok, cnt, end, ln


PROBE_OUT_WORDS = 8192


def stream_read(buf, mode: int = 0, *, out=None, events=None):
    """Read the device tensor `buf` once (int4vh_stream_read): mode 0 loads
    into registers, mode 1 copies into LDS like the verify kernel.  Returns
    the per-wave words (uint32 as int32 [8192]); in mode 0 their xor is the
    xor of the buffer's 32-bit words.  events=(before, after) take the
    kernel's dispatch start and end."""
    if not isinstance(buf, torch.Tensor) or not buf.is_cuda or not buf.is_contiguous():
        raise TypeError("buf must be a contiguous CUDA (HIP) tensor")
    dev = buf.device
    if out is None:
        out = torch.zeros(PROBE_OUT_WORDS, dtype=torch.int32, device=dev)
    nbytes = buf.numel() * buf.element_size()
    stream = torch.cuda.current_stream(dev)
    e0 = _event_handle(events[0], stream) if events else None
    e1 = _event_handle(events[1], stream) if events else None
    st = load_library().int4vh_stream_read(_ptr(buf), nbytes, int(mode), _ptr(out), _stream_ptr(dev), e0, e1)
    if st != OK:
        _raise(st, "int4vh_stream_read")
    return out


# ---------------------------------------------------------------- rows in front of the products

ROWS_F16, ROWS_BF16, ROWS_F32 = 0, 1, 2
_ROW_DTYPES = {torch.float16: ROWS_F16, torch.bfloat16: ROWS_BF16, torch.float32: ROWS_F32}
# A device's current stream by its index, and the current device.  The calls
# behind torch.cuda's take 0.06 us (instead of 1.1) and 0.12 (0.23); where a
# build of torch has not got them, the public ones serve.
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda index: torch.cuda.current_stream(index).cuda_stream))
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())


def _row_code(t, name):
    code = _ROW_DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor of float16, bfloat16 or float32")
    return code


def _on(index, call, *args):
    """A call that launches on the device of that index, made current for it."""
    if index == _current_device():
        return call(*args)
    with torch.cuda.device(index):
        return call(*args)


def _same_device(index, **tensors):
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, not on device {index}")


def _rows2d(t, name):
    """Rows and channels of t [M, H], and the rows' distance in elements; other
    numbers of dims must be contiguous and count as rows of their last."""
    shape = t.shape
    if len(shape) == 2:
        M, H = shape
        stride, inner = t.stride()
        if H > 1 and inner != 1:
            raise ValueError(f"{name} must have contiguous channels")
        if M <= 1:
            stride = H
    else:
        if not shape or not t.is_contiguous():
            raise ValueError(f"{name} must be [M, H], or contiguous with any leading dims")
        stride = H = shape[-1]
        M = t.numel() // H if H else 0
    if M < 1 or H < 1:
        raise ValueError(f"{name} must not be empty")
    if M > 0x7FFFFFFF or H > 0x7FFFFFFF:
        raise ValueError(f"{name} has too many rows or channels")
    if stride < H:
        raise ValueError(f"{name} must not have overlapping rows")
    return M, H, stride


def _vector(t, name, dtype, n):
    """Checks a contiguous vector of n values."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        _check(t, name, dtype, 1)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and hold {n} values")


def _norm_args(x, weight, residual):
    dt = _row_code(x, "x")
    wdt = _row_code(weight, "weight")
    M, H, xs = _rows2d(x, "x")
    if weight.shape != (H,) or not weight.is_contiguous():
        raise ValueError("weight must be contiguous [H]")
    index = x.get_device()
    if weight.get_device() != index:
        _same_device(index, weight=weight)
    if residual is None:
        return dt, wdt, xs, None, 0, None, M, H, index
    if residual.dtype != x.dtype or residual.shape != x.shape:
        raise ValueError("residual must have the type and shape of x")
    rs = _rows2d(residual, "residual")[2]
    if residual.get_device() != index:
        _same_device(index, residual=residual)
    total = torch.empty_like(x, memory_format=torch.contiguous_format)
    return dt, wdt, xs, residual.data_ptr(), rs, total, M, H, index


def rms_norm(x, weight, residual=None, *, eps: float = 1e-6, out_dtype=torch.float16):
    """Root-mean-square norm of rows x [..., H] (float16, bfloat16 or float32;
    a 2-D x may have strided rows), after adding the residual if one is given:
    the hidden states of the verify calls (out_dtype float16).  weight [H].
    Returns the normed rows, and with a residual also the sum x + residual in
    x's type: (normed, sum)."""
    dt, wdt, xs, res, rs, total, M, H, index = _norm_args(x, weight, residual)
    odt = _ROW_DTYPES.get(out_dtype)
    if odt is None:
        raise TypeError("out_dtype must be float16, bfloat16 or float32")
    out = (torch.empty_like(x, memory_format=torch.contiguous_format) if odt == dt
           else x.new_empty(x.shape, dtype=out_dtype))
    st = _on(index, load_library().rms_norm_rows, x.data_ptr(), xs, res, rs, dt, weight.data_ptr(), wdt, M, H, eps,
             None if total is None else total.data_ptr(), out.data_ptr(), odt, _raw_stream(index))
    if st != OK:
        _raise(st, "rms_norm_rows")
    return out if total is None else (out, total)


def rms_norm_int8(x, weight, residual=None, *, channel_scales=None, eps: float = 1e-6):
    """rms_norm with an output in 8 bits, the activations of linear_int4:
    channel_scales (float16 [H]), the per-channel scales of the packed int4
    weights, are folded in.  Returns (codes int8 [..., H], row_scales float32
    [M]), and with a residual also the sum: (codes, row_scales, sum)."""
    dt, wdt, xs, res, rs, total, M, H, index = _norm_args(x, weight, residual)
    cs = None
    if channel_scales is not None:
        _vector(channel_scales, "channel_scales", torch.float16, H)
        _same_device(index, channel_scales=channel_scales)
        cs = channel_scales.data_ptr()
    codes = x.new_empty(x.shape, dtype=torch.int8)
    row_scales = x.new_empty(M, dtype=torch.float32)
    st = _on(index, load_library().rms_norm_rows_int8, x.data_ptr(), xs, res, rs, dt, weight.data_ptr(), wdt, cs, M,
             H, eps, None if total is None else total.data_ptr(), codes.data_ptr(), row_scales.data_ptr(),
             _raw_stream(index))
    if st != OK:
        _raise(st, "rms_norm_rows_int8")
    return (codes, row_scales) if total is None else (codes, row_scales, total)


def quantize_rows(x, *, channel_scales=None):
    """Rows x [..., H] in 8 bits with one scale per row, without a norm (the
    activations of a linear_int4 whose input is no norm; H up to 65536).  Returns (codes int8
    [..., H], row_scales float32 [M])."""
    dt = _row_code(x, "x")
    M, H, xs = _rows2d(x, "x")
    index = x.get_device()
    cs = None
    if channel_scales is not None:
        _vector(channel_scales, "channel_scales", torch.float16, H)
        _same_device(index, channel_scales=channel_scales)
        cs = channel_scales.data_ptr()
    codes = x.new_empty(x.shape, dtype=torch.int8)
    row_scales = x.new_empty(M, dtype=torch.float32)
    st = _on(index, load_library().quantize_rows_int8, x.data_ptr(), xs, dt, cs, M, H, codes.data_ptr(),
             row_scales.data_ptr(), _raw_stream(index))
    if st != OK:
        _raise(st, "quantize_rows_int8")
    return codes, row_scales


_GATES = {None: 0, "sigmoid": 1}


def _norm_weight(w, name, H, index):
    """Address and type of a norm's weight."""
    code = _row_code(w, name)
    if w.shape != (H,) or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous [H]")
    if w.get_device() != index:
        _same_device(index, **{name: w})
    return w.data_ptr(), code


def _block_args(x, residual, post_weight, pre_weight, gate, gate_activation):
    """The leading arguments of both block norms, and (M, H, device index, sum)."""
    dt = _row_code(x, "x")
    M, H, xs = _rows2d(x, "x")
    index = x.get_device()
    if _row_code(residual, "residual") != dt or residual.shape != x.shape:
        raise ValueError("residual must have the type and shape of x")
    rs = _rows2d(residual, "residual")[2]
    if residual.get_device() != index:
        _same_device(index, residual=residual)
    wdt = post = pre = at = None
    if post_weight is not None:
        post, wdt = _norm_weight(post_weight, "post_weight", H, index)
    if pre_weight is not None:
        pre, code = _norm_weight(pre_weight, "pre_weight", H, index)
        if post is not None and wdt != code:
            raise TypeError("post_weight and pre_weight must have one type")
        wdt = code
    act = _GATES.get(gate_activation)
    if act is None:
        raise ValueError("gate_activation must be None or 'sigmoid'")
    gs = 0
    if gate is not None:
        if _row_code(gate, "gate") != dt:
            raise TypeError("gate must have the type of x")
        if gate.shape == x.shape and gate.dim() > 1:
            gs = _rows2d(gate, "gate")[2]
        elif gate.shape != (H,) or not gate.is_contiguous():
            raise ValueError("gate must be contiguous [H], or of the shape of x")
        if gate.get_device() != index:
            _same_device(index, gate=gate)
        at = gate.data_ptr()
    elif act:
        raise ValueError("gate_activation needs a gate")
    total = torch.empty_like(x, memory_format=torch.contiguous_format)
    return (x.data_ptr(), xs, residual.data_ptr(), rs, at, gs, act, dt, post, pre, wdt or 0), M, H, index, total


def rms_norm_block(x, residual, post_weight=None, pre_weight=None, *, gate=None, gate_activation=None,
                   scale: float = 1.0, eps: float = 1e-6, out_dtype=torch.float16):
    """Between two blocks, in one pass: the norm behind the first (post_weight
    [H], or None), its gate and scale, the residual's addition, and the norm in
    front of the second (pre_weight [H], or None):
    sum = residual + x * rstd(x) * post_weight * gate * scale, normed = sum *
    rstd(sum) * pre_weight (from the sum before it is rounded).  x and residual
    [..., H] as in rms_norm; gate: [H], or of the shape of x; gate_activation:
    None or "sigmoid".  Returns (normed of out_dtype, sum in x's type); normed
    is None without pre_weight."""
    args, M, H, index, total = _block_args(x, residual, post_weight, pre_weight, gate, gate_activation)
    odt = _ROW_DTYPES.get(out_dtype)
    if odt is None:
        raise TypeError("out_dtype must be float16, bfloat16 or float32")
    out = None
    if pre_weight is not None:
        out = torch.empty_like(total) if odt == args[7] else torch.empty_like(total, dtype=out_dtype)
    st = _on(index, load_library().rms_norm_block_rows, *args, scale, M, H, eps, total.data_ptr(), _at(out), odt,
             _raw_stream(index))
    if st != OK:
        _raise(st, "rms_norm_block_rows")
    return out, total


def rms_norm_block_int8(x, residual, post_weight, pre_weight, *, gate=None, gate_activation=None, scale: float = 1.0,
                        channel_scales=None, eps: float = 1e-6):
    """rms_norm_block with its output in 8 bits, as rms_norm_int8 gives it:
    (codes int8 [..., H], row_scales float32 [M], sum)."""
    if pre_weight is None:
        raise ValueError("pre_weight is required")
    args, M, H, index, total = _block_args(x, residual, post_weight, pre_weight, gate, gate_activation)
    cs = None
    if channel_scales is not None:
        _vector(channel_scales, "channel_scales", torch.float16, H)
        _same_device(index, channel_scales=channel_scales)
        cs = channel_scales.data_ptr()
    codes = torch.empty_like(total, dtype=torch.int8)
    row_scales = x.new_empty(M, dtype=torch.float32)
    st = _on(index, load_library().rms_norm_block_rows_int8, *args, cs, scale, M, H, eps, total.data_ptr(),
             codes.data_ptr(), row_scales.data_ptr(), _raw_stream(index))
    if st != OK:
        _raise(st, "rms_norm_block_rows_int8")
    return codes, row_scales, total


# ---------------------------------------------------------------- linear layers on packed int4 weights

_ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "silu": 3}


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load_library().linear_int4_rows_workspace_bytes(M, N, K))


def linear_int4(codes, row_scales, packed_w, *, out_scales=None, bias=None, activation=None, residual=None,
                out_dtype=torch.float16, out=None):
    """Linear layer of 8-bit rows (codes int8 [M, K], row_scales float32 [M];
    rms_norm_int8, quantize_rows) on packed int4 weights (uint8 [N, K/2], as
    requant_pack makes them): activation(codes @ q.T * row_scales * out_scales
    + bias) + residual.  out_scales: float32 [N]; bias [N] and residual [M, N]
    of out_dtype; activation: None, "relu", "gelu" or "silu".  out: the [M, N]
    tensor to write, which may be residual itself.  Returns it."""
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda or codes.dtype != torch.int8:
        raise TypeError("codes must be a CUDA (HIP) int8 tensor")
    M, K, cs = _rows2d(codes, "codes")
    _check(packed_w, "packed_w", torch.uint8, 2)
    N = packed_w.shape[0]
    if packed_w.shape[1] * 2 != K:
        raise ValueError("shape mismatch between codes and packed_w")
    _vector(row_scales, "row_scales", torch.float32, M)
    dt = _ROW_DTYPES.get(out_dtype)
    if dt is None:
        raise TypeError("out_dtype must be float16, bfloat16 or float32")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be None, 'relu', 'gelu' or 'silu'")
    if out_scales is not None:
        _vector(out_scales, "out_scales", torch.float32, N)
    if bias is not None:
        _vector(bias, "bias", out_dtype, N)
    index = codes.get_device()
    rs, os_ = 0, N
    shape = codes.shape[:-1] + (N,)
    if residual is not None:
        if _row_code(residual, "residual") != dt or residual.shape != shape:
            raise ValueError("residual must be [M, N] of out_dtype")
        rs = _rows2d(residual, "residual")[2]
    if out is None:
        out = row_scales.new_empty(shape, dtype=out_dtype)
    else:
        if _row_code(out, "out") != dt or out.shape != shape:
            raise ValueError("out must be [M, N] of out_dtype")
        os_ = _rows2d(out, "out")[2]
    _same_device(index, row_scales=row_scales, packed_w=packed_w, out_scales=out_scales, bias=bias, residual=residual,
                 out=out)
    st = _on(index, _launch_linear, index, codes.data_ptr(), cs, row_scales, packed_w.data_ptr(), _at(out_scales),
             _at(bias), act, _at(residual), rs, M, N, K, out.data_ptr(), os_, dt)
    if st != OK:
        _raise(st, "linear_int4_rows")
    return out


def _launch_linear(index, codes, cs, row_scales, packed_w, out_scales, bias, act, residual, rs, M, N, K, out, os_, dt):
    L = load_library()
    need = L.linear_int4_rows_workspace_bytes(M, N, K)
    ws = row_scales.new_empty(need, dtype=torch.uint8) if need else None
    return L.linear_int4_rows(codes, cs, row_scales.data_ptr(), packed_w, out_scales, bias, act, residual, rs, M, N, K,
                              out, os_, dt, _at(ws), need, _raw_stream(index))


def _at(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------- 4-bit floating point

def quantize_mxfp4(x):
    """Rows x [..., H] (float16, bfloat16 or float32; H a multiple of 32 up to
    65536) in microscaled 4-bit floating point, one power of two for 32
    channels: activations and weights of linear_mxfp4 alike.  Returns (codes
    uint8 [..., H/2], the even channel in the low half of a byte, and scales
    uint8 [..., H/32], exponents + 127)."""
    dt = _row_code(x, "x")
    M, H, xs = _rows2d(x, "x")
    if H % 32:
        raise ValueError("the channels of x must be a multiple of 32")
    index = x.get_device()
    lead = x.shape[:-1]
    codes = x.new_empty(lead + (H // 2,), dtype=torch.uint8)
    scales = x.new_empty(lead + (H // 32,), dtype=torch.uint8)
    st = _on(index, load_library().quantize_rows_mxfp4, x.data_ptr(), xs, dt, M, H, codes.data_ptr(),
             scales.data_ptr(), _raw_stream(index))
    if st != OK:
        _raise(st, "quantize_rows_mxfp4")
    return codes, scales


def _mx_rows(codes, scales, names=("codes", "scales")):
    """(M, K) of a matrix in 4-bit floating point."""
    if (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and codes.dim() == 2 and codes.is_cuda
            and scales.is_cuda and codes.dtype == scales.dtype == torch.uint8 and codes.is_contiguous()
            and scales.is_contiguous()):
        M, half = codes.shape                  # the usual matrix
        if 1 <= M <= 0x7FFFFFFF and half >= 16 and half % 16 == 0 and scales.shape == (M, half // 16):
            return M, 2 * half
    for t, name in ((codes, names[0]), (scales, names[1])):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.uint8:
            raise TypeError(f"{name} must be a CUDA (HIP) uint8 tensor")
        if not t.dim() or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous rows")
    K = 2 * codes.shape[-1]
    if K < 32 or K % 32 or scales.shape != codes.shape[:-1] + (K // 32,):
        raise ValueError(f"{names[1]} must hold one byte for 32 channels of {names[0]}")
    M = codes.numel() // (K // 2)
    if M < 1 or M > 0x7FFFFFFF:
        raise ValueError(f"{names[0]} must have between 1 and 2^31 - 1 rows")
    return M, K


def dequantize_mxfp4(codes, scales, *, out_dtype=torch.float16):
    """The values of rows in 4-bit floating point (quantize_mxfp4): codes
    [..., H/2], scales [..., H/32] -> [..., H] of out_dtype."""
    M, H = _mx_rows(codes, scales)
    dt = _ROW_DTYPES.get(out_dtype)
    if dt is None:
        raise TypeError("out_dtype must be float16, bfloat16 or float32")
    index = codes.get_device()
    if scales.get_device() != index:
        _same_device(index, scales=scales)
    out = codes.new_empty(codes.shape[:-1] + (H,), dtype=out_dtype)
    st = _on(index, load_library().dequantize_rows_mxfp4, codes.data_ptr(), scales.data_ptr(), M, H, out.data_ptr(),
             dt, _raw_stream(index))
    if st != OK:
        _raise(st, "dequantize_rows_mxfp4")
    return out


def linear_mxfp4_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load_library().linear_mxfp4_rows_workspace_bytes(M, N, K))


def linear_mxfp4(codes, scales, w_codes, w_scales, *, bias=None, activation=None, residual=None,
                 out_dtype=torch.float16, out=None):
    """Linear layer between two matrices in 4-bit floating point
    (quantize_mxfp4): rows codes [..., K/2], scales [..., K/32] and weights
    w_codes [N, K/2], w_scales [N, K/32]: activation(x @ w.T + bias) +
    residual.  bias [N] and residual [..., N] of out_dtype; activation: None,
    "relu", "gelu" or "silu".  out: the [..., N] tensor to write, which may be
    residual itself.  Returns it."""
    M, K = _mx_rows(codes, scales)
    if w_codes.dim() != 2:
        raise ValueError("w_codes must be [N, K/2]")
    N, wk = _mx_rows(w_codes, w_scales, ("w_codes", "w_scales"))
    if wk != K:
        raise ValueError("shape mismatch between codes and w_codes")
    dt = _ROW_DTYPES.get(out_dtype)
    if dt is None:
        raise TypeError("out_dtype must be float16, bfloat16 or float32")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be None, 'relu', 'gelu' or 'silu'")
    if bias is not None:
        _vector(bias, "bias", out_dtype, N)
    index = codes.get_device()
    rs, os_ = 0, N
    shape = codes.shape[:-1] + (N,)
    if residual is not None:
        if _row_code(residual, "residual") != dt or residual.shape != shape:
            raise ValueError("residual must be [..., N] of out_dtype")
        rs = _rows2d(residual, "residual")[2]
    if out is None:
        out = codes.new_empty(shape, dtype=out_dtype)
    else:
        if _row_code(out, "out") != dt or out.shape != shape:
            raise ValueError("out must be [..., N] of out_dtype")
        os_ = _rows2d(out, "out")[2]
    for t in (scales, w_codes, w_scales, bias, residual, out):
        if t is not None and t.get_device() != index:
            _same_device(index, scales=scales, w_codes=w_codes, w_scales=w_scales, bias=bias, residual=residual,
                         out=out)
    st = _on(index, _launch_linear_mxfp4, index, codes, scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(),
             _at(bias), act, _at(residual), rs, M, N, K, out.data_ptr(), os_, dt)
    if st != OK:
        _raise(st, "linear_mxfp4_rows")
    return out


def _launch_linear_mxfp4(index, codes, scales, w_codes, w_scales, bias, act, residual, rs, M, N, K, out, os_, dt):
    L = load_library()
    need = L.linear_mxfp4_rows_workspace_bytes(M, N, K)
    ws = codes.new_empty(need) if need else None
    return L.linear_mxfp4_rows(codes.data_ptr(), scales, w_codes, w_scales, bias, act, residual, rs, M, N, K, out, os_,
                               dt, _at(ws), need, _raw_stream(index))


# ---------------------------------------------------------------- rules on logits

_RULES = struct.Struct("@PqPPPPPPPqPPqqP")     # int4vh_logit_rules


class LogitRules:
    """Penalties for repeated tokens, biases and grammar masks of R requests
    (int4vh_logits.h), every part optional; device tensors, kept by reference.
    history int32 [total] (the requests' tokens back to back, prompt first),
    history_offsets int64 [R+1], n_prompt int32 [R]; repetition, frequency,
    presence float32 [R]; bias_ids int32 and bias_values float32 [n],
    bias_offsets int64 [R+1] (the last of entries with one id holds); mask
    int32 [n, >= ceil(V/32)], bit v % 32 of word v // 32 set where token v is
    allowed, and mask_index int32 [R*T], each row's mask (negative: the row is
    free; without it row r has mask r)."""

    __slots__ = ("device", "tensors", "packed", "requests", "mask_rows", "mask_words", "n_index")

    def __init__(self, *, history=None, history_offsets=None, n_prompt=None, repetition=None, frequency=None,
                 presence=None, bias_ids=None, bias_values=None, bias_offsets=None, mask=None, mask_index=None):
        self.device = self.requests = self.n_index = None
        self.tensors = (history, history_offsets, n_prompt, repetition, frequency, presence, bias_ids, bias_values,
                        bias_offsets, mask, mask_index)
        place = self._place
        n_history = n_bias = 0
        p_history = p_offsets = p_prompt = p_rep = p_freq = p_pres = p_ids = p_values = p_boffsets = 0
        if history is not None:
            if history_offsets is None:
                raise ValueError("history and history_offsets go together")
            p_history, n_history = place(history, "history", torch.int32), history.shape[0]
            p_offsets = place(history_offsets, "history_offsets", torch.int64, 1)
        elif history_offsets is not None or n_prompt is not None:
            raise ValueError("history_offsets and n_prompt need a history")
        if n_prompt is not None:
            p_prompt = place(n_prompt, "n_prompt", torch.int32, 0)
        if repetition is not None:
            p_rep = place(repetition, "repetition", torch.float32, 0)
        if frequency is not None:
            p_freq = place(frequency, "frequency", torch.float32, 0)
        if presence is not None:
            p_pres = place(presence, "presence", torch.float32, 0)
        if bias_ids is not None and bias_values is not None and bias_offsets is not None:
            p_ids, n_bias = place(bias_ids, "bias_ids", torch.int32), bias_ids.shape[0]
            p_values = place(bias_values, "bias_values", torch.float32)
            p_boffsets = place(bias_offsets, "bias_offsets", torch.int64, 1)
            if bias_values.shape[0] != n_bias:
                raise ValueError("bias_ids and bias_values must have one length")
        elif bias_ids is not None or bias_values is not None or bias_offsets is not None:
            raise ValueError("bias_ids, bias_values and bias_offsets go together")
        stride = p_mask = p_index = 0
        self.mask_rows = self.mask_words = 0
        if mask is not None:
            if not isinstance(mask, torch.Tensor) or not mask.is_cuda or mask.dtype != torch.int32 or mask.dim() != 2:
                raise TypeError("mask must be a 2-D int32 CUDA (HIP) tensor")
            self.mask_rows, self.mask_words, stride = _rows2d(mask, "mask")
            self._on(mask, "mask")
            p_mask = mask.data_ptr()
            if mask_index is not None:
                p_index, self.n_index = place(mask_index, "mask_index", torch.int32), mask_index.shape[0]
        elif mask_index is not None:
            raise ValueError("mask_index needs a mask")
        self.packed = _RULES.pack(p_history, n_history, p_offsets, p_prompt, p_rep, p_freq, p_pres, p_ids, p_values,
                                  n_bias, p_boffsets, p_mask, self.mask_rows, stride, p_index)

    def _place(self, t, name, dtype, extra=None):
        """Checks a contiguous vector, one value per request (and `extra`) where
        that is given, and returns its address."""
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or t.dim() != 1 or not t.is_contiguous():
            _check(t, name, dtype, 1)
        self._on(t, name)
        if extra is not None:
            n = t.shape[0] - extra
            if self.requests is None:
                self.requests = n
            elif self.requests != n:
                raise ValueError(f"{name} is for {n} requests, not {self.requests}")
        return t.data_ptr()

    def _on(self, t, name):
        index = t.get_device()
        if self.device is None:
            self.device = index
        elif index != self.device:
            raise ValueError(f"{name} is on device {index}, not on {self.device}")

    def check(self, index, R, T, V):
        """Raises unless the rules fit a call of these sizes on that device."""
        if self.device is not None and self.device != index:
            raise ValueError(f"the rules are on device {self.device}, not on {index}")
        if self.requests is not None and self.requests != R:
            raise ValueError(f"the rules are for {self.requests} requests, not {R}")
        if self.mask_rows:
            if self.mask_words < (V + 31) // 32:
                raise ValueError("mask must hold a bit per token")
            if self.n_index is not None and self.n_index != R * T:
                raise ValueError("mask_index must hold one index per row")
            if self.n_index is None and self.mask_rows != R * T:
                raise ValueError("mask must hold one row per row of the logits, or come with mask_index")


def _logit_rows(logits, R):
    """(type code, rows' distance, R, T, V) of logits [R, T, V], or [R*T, V]
    with R."""
    code = _row_code(logits, "logits")
    if logits.dim() == 3:
        if R is not None and R != logits.shape[0]:
            raise ValueError("R does not match the logits")
        R = logits.shape[0]
    elif logits.dim() != 2:
        raise ValueError("logits must be [R, T, V], or [R*T, V] with R")
    elif R is None:
        raise ValueError("R is required for 2-D logits")
    M, V, stride = _rows2d(logits, "logits")
    if R < 1 or M % R:
        raise ValueError("the logits' rows must be R*T")
    return code, stride, R, M // R, V


def _drafted(t, name, dtype, n, index):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        _check(t, name, dtype)
    if t.numel() != n:
        raise ValueError(f"{name} must hold R*(T-1) values")
    if t.get_device() != index:
        _same_device(index, **{name: t})
    return t.data_ptr()


def _drafts(index, R, T, draft_ids, draft_probs=None, uniforms=None):
    if T == 1:
        return None, None, None
    if draft_ids is None:
        raise ValueError("draft_ids is required when T > 1")
    n = R * (T - 1)
    ids = _drafted(draft_ids, "draft_ids", torch.int32, n, index)
    if draft_probs is None and uniforms is None:
        return ids, None, None
    if draft_probs is None or uniforms is None:
        raise ValueError("draft_probs and uniforms go together")
    return (ids, _drafted(draft_probs, "draft_probs", torch.float32, n, index),
            _drafted(uniforms, "uniforms", torch.float32, n, index))


def apply_logit_rules(logits, rules, draft_ids=None, *, R: int | None = None, out=None):
    """The logits under the rules (LogitRules), written out: logits [R, T, V],
    or [R*T, V] with R (float32, float16 or bfloat16; 2-D rows may be
    strided); draft_ids int32 [R, T-1] (None when T == 1): row t counts drafts
    0 .. t-1 as generated.  out: the tensor to write, of the logits' shape and
    type, which may be the logits.  Returns it."""
    code, stride, R, T, V = _logit_rows(logits, R)
    index = logits.get_device()
    if rules is not None:
        rules.check(index, R, T, V)
    dr = _drafts(index, R, T, draft_ids)[0]
    os_ = V
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    else:
        if not isinstance(out, torch.Tensor) or out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out must have the shape and type of the logits")
        _same_device(index, out=out)
        os_ = _rows2d(out, "out")[2]
    st = _on(index, load_library().logit_rules_apply, logits.data_ptr(), stride, code, dr, R, T, V,
             None if rules is None else rules.packed, out.data_ptr(), os_, _raw_stream(index))
    if st != OK:
        _raise(st, "logit_rules_apply")
    return out


def _verify_outputs(like, M, R, T, k, sampled, want_lse):
    f, i, new = torch.float32, torch.int32, like.new_empty
    return (new(M, dtype=f), new(M, dtype=i), new((M, k), dtype=i) if k else None, new((M, k), dtype=f) if k else None,
            new((R, T - 1), dtype=f) if sampled else None, new(R, dtype=i), new(M, dtype=f) if want_lse else None)


def verify_logits(logits, rules=None, draft_ids=None, draft_probs=None, uniforms=None, *, top_k: int = 0,
                  temperature: float = 1.0, R: int | None = None, want_lse: bool = False):
    """Verification of drafted tokens straight from logits [R, T, V] (or [R*T,
    V] with R) under rules (LogitRules, or None), in one pass over them.
    With draft_probs and uniforms (float32 [R, T-1]) as verify_sampled: top-k
    sampling at a temperature, or over the whole vocabulary (top_k == 0);
    without them the drafts are verified greedily, as verify_batch does.
    Returns (logits_max [R*T], argmax_ids [R*T], topk_ids [R*T, k], topk_logits
    [R*T, k], p_draft [R, T-1], n_accepted [R], lse [R*T]); the top-k outputs
    are None when top_k == 0, p_draft without draft_probs or when T == 1, lse
    unless want_lse.  A row whose mask leaves nothing has argmax -1."""
    code, stride, R, T, V = _logit_rows(logits, R)
    index = logits.get_device()
    if rules is not None:
        rules.check(index, R, T, V)
    dr, dp, un = _drafts(index, R, T, draft_ids, draft_probs, uniforms)
    M, k = R * T, int(top_k)
    L = load_library()
    need = L.logit_rules_verify_workspace_bytes(R, T, V, k)
    if need == 0:
        _raise(EINVAL, "logit_rules_verify")
    out = lmax, amax, tids, tlog, pdr, nacc, lse = _verify_outputs(logits, M, R, T, k, dp is not None, want_lse)
    ws = logits.new_empty(need, dtype=torch.uint8)
    st = _on(index, L.logit_rules_verify, logits.data_ptr(), stride, code, dr, dp, un, R, T, V,
             None if rules is None else rules.packed, k, temperature, lmax.data_ptr(), amax.data_ptr(), _at(tids),
             _at(tlog), _at(lse), _at(pdr), nacc.data_ptr(), ws.data_ptr(), need, _raw_stream(index))
    if st != OK:
        _raise(st, "logit_rules_verify")
    return out


def verify_ruled(hidden, packed_w, scales, rules, draft_ids=None, draft_probs=None, uniforms=None, *,
                 top_k: int = 0, temperature: float = 1.0, R: int | None = None, want_lse: bool = False,
                 workspace: Workspace | None = None):
    """Verification through the head under rules (LogitRules): verify_batch's
    logits through verify_logits, in one call.  hidden: float16 [R, T, H] (or
    [R*T, H] with R); the other arguments and the outputs as verify_logits.
    The workspace also holds the call's logits, R*T*V*4 bytes
    (verify_lm_head_int4_ruled_workspace_bytes); without one of the caller's,
    the stream's own grows to that size and is kept for later calls."""
    if hidden.dim() == 3:
        R, T, H = hidden.shape
        hidden = hidden.reshape(R * T, H)
    else:
        if R is None:
            raise ValueError("R is required for a 2-D hidden tensor")
        T = hidden.shape[0] // R
        H = hidden.shape[1]
    _check(hidden, "hidden", torch.float16, 2)
    _check(packed_w, "packed_w", torch.uint8, 2)
    _check(scales, "scales", torch.float16, 1)
    V = packed_w.shape[0]
    if packed_w.shape[1] * 2 != H or scales.shape[0] != H or hidden.shape[0] != R * T:
        raise ValueError("shape mismatch between hidden, packed_w and scales")
    index = hidden.get_device()
    _same_device(index, packed_w=packed_w, scales=scales)
    if rules is not None:
        rules.check(index, R, T, V)
    dr, dp, un = _drafts(index, R, T, draft_ids, draft_probs, uniforms)
    k = int(top_k)
    L = load_library()
    need = L.verify_lm_head_int4_ruled_workspace_bytes(R, T, V, H, k)
    if need == 0:
        _raise(EINVAL, "verify_lm_head_int4_ruled")
    out = lmax, amax, tids, tlog, pdr, nacc, lse = _verify_outputs(hidden, R * T, R, T, k, dp is not None, want_lse)
    if workspace is None:
        workspace = _on(index, _default_workspace, hidden.device, need)
    else:
        _same_device(index, workspace=workspace.tensor)
    st = _on(index, L.verify_lm_head_int4_ruled, hidden.data_ptr(), packed_w.data_ptr(), scales.data_ptr(), dr, dp, un,
             R, T, V, H, None if rules is None else rules.packed, k, temperature, lmax.data_ptr(), amax.data_ptr(),
             _at(tids), _at(tlog), _at(lse), _at(pdr), nacc.data_ptr(), workspace.tensor.data_ptr(), workspace.nbytes,
             _raw_stream(index))
    if st != OK:
        _raise(st, "verify_lm_head_int4_ruled")
    return out


# ---------------------------------------------------------------- sampling

_SAMPLING = struct.Struct("@PPPPfiff")     # int4vh_sampling


def sample_workspace_bytes(R: int, T: int, V: int) -> int:
    return int(load_library().sample_logits_workspace_bytes(R, T, V))


def _setting(v, name, dtype, R, index):
    """(device address or 0, scalar) of a setting: a number, or a tensor [R]."""
    if isinstance(v, torch.Tensor):
        if v.dtype != dtype or not v.is_cuda or v.shape != (R,) or not v.is_contiguous():
            _vector(v, name, dtype, R)
        if v.get_device() != index:
            _same_device(index, **{name: v})
        return v.data_ptr(), 0
    return 0, v


def sample_logits(logits, uniforms, rules=None, draft_ids=None, *, R: int | None = None, temperature=1.0, top_k=0,
                  top_p=1.0, min_p=0.0, accept=None):
    """A token of every row of logits [R, T, V] (or [R*T, V] with R; float32,
    float16 or bfloat16), drawn by uniforms (float32, R*T numbers in [0, 1)) at
    a temperature among the top_k best (0: all), of these the best that hold
    top_p of the mass, and of these those with at least min_p of the best one's
    mass, under rules (LogitRules, or None; draft_ids int32 [R, T-1] when T >
    1, as in verify_logits).  temperature, top_p, min_p: numbers, or float32
    [R], and top_k a number, or int32 [R], a value per request; a temperature of 0
    takes the best token.  With accept (float32 [R, T-1], the drafts' own uniform
    numbers) the drafts are verified as point masses: a draft is accepted where
    accept < p_draft, and the tokens of rows with a draft are drawn from the
    others, so that row n_accepted's is the token behind the accepted drafts.
    Returns (token_ids int32 [R*T], -1 for a row that has none, token_probs
    float32 [R*T], p_draft [R, T-1], n_accepted int32 [R]); the last two are
    None without accept."""
    code, stride, R, T, V = _logit_rows(logits, R)
    index = logits.get_device()
    if rules is not None:
        rules.check(index, R, T, V)
    dr = _drafts(index, R, T, draft_ids)[0]
    M = R * T
    if not isinstance(uniforms, torch.Tensor) or uniforms.dtype != torch.float32 or not uniforms.is_cuda:
        _check(uniforms, "uniforms", torch.float32)
    if uniforms.numel() != M or not uniforms.is_contiguous():
        raise ValueError("uniforms must be contiguous and hold R*T values")
    if uniforms.get_device() != index:
        _same_device(index, uniforms=uniforms)
    f, i = torch.float32, torch.int32
    (pt, t), (pk, k), (pp, p), (pm, m) = (_setting(temperature, "temperature", f, R, index),
                                          _setting(top_k, "top_k", i, R, index), _setting(top_p, "top_p", f, R, index),
                                          _setting(min_p, "min_p", f, R, index))
    if not isinstance(k, int):
        raise TypeError("top_k must be a whole number or an int32 tensor")
    settings = _SAMPLING.pack(pt, pk, pp, pm, t, min(max(k, -1), V), p, m)
    new = logits.new_empty
    probs = torch.empty_like(uniforms) if uniforms.dim() == 1 else new(M, dtype=f)
    ids = torch.empty_like(probs, dtype=i)
    ac = pdr = nacc = None
    if accept is not None:
        if T == 1:
            raise ValueError("accept needs drafts")
        ac = _drafted(accept, "accept", f, R * (T - 1), index)
        pdr, nacc = new((R, T - 1), dtype=f), new(R, dtype=i)
    L = load_library()
    need = L.sample_logits_workspace_bytes(R, T, V)
    if need == 0:
        _raise(EINVAL, "sample_logits_rows")
    ws = new(need, dtype=torch.uint8)
    st = _on(index, L.sample_logits_rows, logits.data_ptr(), stride, code, dr, R, T, V,
             None if rules is None else rules.packed, settings, uniforms.data_ptr(), ac, ids.data_ptr(),
             probs.data_ptr(), _at(pdr), _at(nacc), ws.data_ptr(), need, _raw_stream(index))
    if st != OK:
        _raise(st, "sample_logits_rows")
    return ids, probs, pdr, nacc
