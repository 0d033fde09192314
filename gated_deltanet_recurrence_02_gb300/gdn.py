"""ctypes binding of libgdn (include/gdn.h): argument marshalling only.

Every entry point keeps its C name.  Tensors are torch CUDA tensors (the
library only sees their device pointers); shapes give the head counts and
head sizes; the stream defaults to torch's current stream.  Outputs the caller
does not pass are allocated here with torch (device memory is the only thing
torch provides on this path).  Every step of the computation runs in the
library's CUDA kernels; there is no other implementation to fall back to, so
a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import build as _build

GDN_OK, GDN_ERR_WORKSPACE = 0, 7
GDN_F32, GDN_F16, GDN_BF16 = 0, 1, 2
GDN_DEVERR_BAD_INDEX, GDN_DEVERR_TIMEOUT = 1, 2
# input conventions (include/gdn.h): OR'd into dtype_qkv / dtype_gate
GDN_QK_L2NORM, GDN_ALPHA_LOG, GDN_BETA_LOGIT = 0x100, 0x200, 0x400
GDN_ALPHA_PER_HEAD = 0x800
# gates of the norms
GDN_GATE_NONE, GDN_GATE_SILU, GDN_GATE_SIGMOID = 0, 1, 2
GDN_GATE_FIRST, GDN_NORM_UNIT_OFFSET = 0x10, 0x20
# rotation and cached attention
GDN_ROTARY_PAIRS, GDN_ROTARY_INVERSE = 0x1, 0x2
GDN_ATTENTION_FULL = 0x1
_DT = {torch.float32: GDN_F32, torch.float16: GDN_F16, torch.bfloat16: GDN_BF16}

_lib = None


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded libgdn.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(
            f"libgdn.so is not built ({path}); run "
            "`python -c 'import __graft_entry__ as g; g.build()'` first")
    L = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.gdn_prefill_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i]
    L.gdn_prefill_workspace_size.restype = sz
    L.gdn_prefill_chunked.argtypes = [vp] * 8 + [i, vp, vp] + [i] * 8 + [f, i, i, vp, sz, vp]
    L.gdn_prefill_chunked.restype = i
    L.gdn_prefill_chunked_checkpoints.argtypes = ([vp] * 8 + [i, vp, vp] + [i] * 8 + [f, i, i]
                                                  + [vp, i, i, vp, sz, vp])
    L.gdn_prefill_chunked_checkpoints.restype = i
    L.gdn_prefill_chunked_capture.argtypes = ([vp] * 8 + [i, vp, vp] + [i] * 8 + [f, i, i]
                                              + [i, vp, vp, vp, vp, sz, vp])
    L.gdn_prefill_chunked_capture.restype = i
    L.gdn_recurrent_capture.argtypes = ([vp] * 8 + [i, vp, vp] + [i] * 7 + [f, i, i]
                                        + [i, vp, vp, vp, vp])
    L.gdn_recurrent_capture.restype = i
    L.gdn_replay_state_updates.argtypes = [vp, vp, vp, i, vp, i, i, i, i, i, vp]
    L.gdn_replay_state_updates.restype = i
    L.gdn_replay_verify.argtypes = ([vp] * 9 + [i] + [vp] * 3 + [i] * 7 + [f, i, i, i]
                                    + [vp] * 4)
    L.gdn_replay_verify.restype = i
    L.gdn_linear_prefill_workspace_size.argtypes = [i] * 8
    L.gdn_linear_prefill_workspace_size.restype = sz
    L.gdn_linear_prefill.argtypes = [vp] * 7 + [i, vp, vp] + [i] * 7 + [f, i, i, vp, sz, vp]
    L.gdn_linear_prefill.restype = i
    L.gdn_linear_recurrent.argtypes = ([vp] * 7 + [i, vp, vp] + [i] * 7 + [f, i, i]
                                       + [i, vp, vp, vp, vp])
    L.gdn_linear_recurrent.restype = i
    i64 = ctypes.c_int64
    L.gdn_gated_norm.argtypes = [vp] * 4 + [i64, i, i, i64, i64, i64, f, i, i, i, vp]
    L.gdn_gated_norm.restype = i
    L.gdn_residual_norm.argtypes = [vp] * 7 + [i64, i, i64, i64, f, f, i, i, i, i, vp]
    L.gdn_residual_norm.restype = i
    L.gdn_accept_drafts.argtypes = [vp] * 7 + [i, i, i, i64, i64, i, vp]
    L.gdn_accept_drafts.restype = i
    L.gdn_rotary.argtypes = [vp] * 5 + [i64, i, i, i, i, i64, i64, i, i, vp]
    L.gdn_rotary.restype = i
    L.gdn_paged_append.argtypes = ([vp] * 12 + [i] * 7 + [i64] * 4 + [i] * 3 + [i64] * 3 + [i, i, vp])
    L.gdn_paged_append.restype = i
    L.gdn_paged_attention_workspace_size.argtypes = [i] * 7
    L.gdn_paged_attention_workspace_size.restype = sz
    L.gdn_paged_attention.argtypes = ([vp] * 8 + [i] * 5 + [i64] + [i] * 3 + [i64] * 3 + [f, i, i, i, vp, sz, vp])
    L.gdn_paged_attention.restype = i
    L.gdn_device_errors.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    L.gdn_device_errors.restype = i
    L.gdn_status_string.argtypes = [i]
    L.gdn_status_string.restype = ctypes.c_char_p
    L.gdn_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.gdn_set_wait_limit_ns.restype = None
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().gdn_status_string(int(status)).decode()


def _p(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libgdn takes contiguous tensors")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (2.8 us less a
# call on the GB300's host, where a whole decode call takes some ten); the public
# call where this PyTorch has no such function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _empty(shape, dtype, device, stream, scratch: bool = False):
    """Memory for a call on `stream`.  Where that is not the current stream it comes from
    that stream's pool, as for torch operations under torch.cuda.stream: from the current
    one's it could still be in use there, and would be handed out again there as soon as
    the caller drops it, with the call still to run.  What the caller receives (all but
    scratch) is marked as used on the current stream, where it will be read."""
    if stream is None or _stream(stream) == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if not scratch:
        t.record_stream(current)
    return t


# Workspaces that a thread keeps for its calls on the default stream, by device: (tensor,
# pointer, bytes).  The default stream runs them one after the other, is never captured and
# never ends; and another thread's calls, whose launches might come in between, have one of
# their own.  (An allocation behind a launch takes 5 to 7 us of the GB300's host, the rest of
# an attention call 12.)  Calls on other streams allocate.  It is as large as the thread's
# largest such call needed, on a GB300 0.3 to 40 MB (fp32 single tokens; 16-bit chunks), and
# stays until the thread ends; for calls that are given a workspace none is kept.
_kept = threading.local()


def _keep(nbytes: int, device):
    """Make the thread's workspace on the default stream of the current device one of nbytes."""
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    kept = _kept.__dict__[_device()] = (t, t.data_ptr(), nbytes)
    return kept


def _codes(q, alpha, conventions: int):
    """dtype_qkv and dtype_gate arguments: storage types plus the input
    convention bits (GDN_QK_L2NORM goes with q/k, the gate bits with alpha/beta)."""
    return (_DT[q.dtype] | (conventions & GDN_QK_L2NORM),
            _DT[alpha.dtype] | (conventions & (GDN_ALPHA_LOG | GDN_BETA_LOGIT)))


def _check(status: int, where: str):
    if status != GDN_OK:
        raise GdnError(status, where)


def slot_width(Hk: int, Hv: int, dk: int, dv: int) -> int:
    """Floats per captured token: Hv decays, Hk*dk keys, Hv*dv deltas."""
    return Hv + Hk * dk + Hv * dv


def gdn_prefill_workspace_size(B, T, Hk, Hv, dk, dv, chunk, dtype_qkv, varlen=False) -> int:
    return int(lib().gdn_prefill_workspace_size(B, T, Hk, Hv, dk, dv, chunk,
                                                _DT.get(dtype_qkv, dtype_qkv), int(bool(varlen))))


def _dims(q, v, B, T, cu_seqlens):
    total_T, Hk, dk = q.shape
    _, Hv, dv = v.shape
    if cu_seqlens is None and T is None:
        T = total_T // B if B else 0
    if cu_seqlens is not None:
        T = total_T
    return int(T), int(Hk), int(dk), int(Hv), int(dv)


def gdn_prefill_chunked(q, k, v, alpha, beta, *, B: int, T: Optional[int] = None,
                        cu_seqlens=None, initial_state=None,
                        initial_state_indices=None, final_state=None, out=None,
                        chunk: int = 64, scale: float = 1.0, workspace=None,
                        want_final_state: bool = True, conventions: int = 0, stream=None):
    """Chunked prefill.  Returns (out, final_state)."""
    T, Hk, dk, Hv, dv = _dims(q, v, B, T, cu_seqlens)
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if final_state is None and want_final_state:
        final_state = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    n0 = initial_state.shape[0] if initial_state is not None else 0
    need = gdn_prefill_workspace_size(B, T, Hk, Hv, dk, dv, chunk, q.dtype,
                                      varlen=cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, v.device, stream, scratch=True)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gdn_prefill_chunked(
        _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), _p(initial_state),
        _p(initial_state_indices), n0, _p(final_state), _p(out), B, T, Hk, Hk, Hv,
        dk, dv, chunk, scale, *_codes(q, alpha, conventions), _p(workspace),
        ws_bytes, _stream(stream))
    _check(st, "gdn_prefill_chunked")
    return out, final_state


def gdn_prefill_chunked_checkpoints(q, k, v, alpha, beta, *, B: int, checkpoint_capacity: int,
                                    checkpoint_interval: int = 1, T: Optional[int] = None,
                                    cu_seqlens=None, initial_state=None,
                                    initial_state_indices=None, final_state=None, out=None,
                                    checkpoints=None, chunk: int = 64, scale: float = 1.0,
                                    workspace=None, want_final_state: bool = True,
                                    conventions: int = 0, stream=None):
    """Chunked prefill that also writes the state every checkpoint_interval
    chunks.  Returns (out, final_state, checkpoints [B, capacity, Hv, dv, dk])."""
    T, Hk, dk, Hv, dv = _dims(q, v, B, T, cu_seqlens)
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if final_state is None and want_final_state:
        final_state = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    cap = int(checkpoint_capacity)
    if checkpoints is None and cap > 0:
        checkpoints = _empty((B, cap, Hv, dv, dk), torch.float32, v.device, stream)
    n0 = initial_state.shape[0] if initial_state is not None else 0
    need = gdn_prefill_workspace_size(B, T, Hk, Hv, dk, dv, chunk, q.dtype,
                                      varlen=cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, v.device, stream, scratch=True)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gdn_prefill_chunked_checkpoints(
        _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), _p(initial_state),
        _p(initial_state_indices), n0, _p(final_state), _p(out), B, T, Hk, Hk, Hv,
        dk, dv, chunk, scale, *_codes(q, alpha, conventions), _p(checkpoints), cap,
        int(checkpoint_interval), _p(workspace), ws_bytes, _stream(stream))
    _check(st, "gdn_prefill_chunked_checkpoints")
    return out, final_state, checkpoints


def gdn_prefill_chunked_capture(q, k, v, alpha, beta, *, B: int, state_update_capacity: int,
                                capture_count, T: Optional[int] = None, cu_seqlens=None,
                                initial_state=None, initial_state_indices=None,
                                final_state=None, out=None, state_update_active=None,
                                state_update=None, chunk: int = 64, scale: float = 1.0,
                                workspace=None, want_final_state: bool = True,
                                conventions: int = 0, stream=None):
    """Chunked prefill with the compact capture of gdn_recurrent_capture.
    Returns (out, final_state, state_update)."""
    T, Hk, dk, Hv, dv = _dims(q, v, B, T, cu_seqlens)
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if final_state is None and want_final_state:
        final_state = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    cap = int(state_update_capacity)
    if cap > 0 and state_update is None:
        state_update = _empty((B, cap, slot_width(Hk, Hv, dk, dv)), torch.float32, v.device,
                              stream)
    n0 = initial_state.shape[0] if initial_state is not None else 0
    need = gdn_prefill_workspace_size(B, T, Hk, Hv, dk, dv, chunk, q.dtype,
                                      varlen=cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, v.device, stream, scratch=True)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gdn_prefill_chunked_capture(
        _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), _p(initial_state),
        _p(initial_state_indices), n0, _p(final_state), _p(out), B, T, Hk, Hk, Hv,
        dk, dv, chunk, scale, *_codes(q, alpha, conventions), cap, _p(capture_count),
        _p(state_update_active), _p(state_update), _p(workspace), ws_bytes, _stream(stream))
    _check(st, "gdn_prefill_chunked_capture")
    return out, final_state, state_update


def gdn_recurrent_capture(q, k, v, alpha, beta, *, B: int, T: Optional[int] = None,
                          cu_seqlens=None, initial_state=None,
                          initial_state_indices=None, final_state=None, out=None,
                          scale: float = 1.0, state_update_capacity: int = 0,
                          capture_count=None, state_update_active=None,
                          state_update=None, want_final_state: bool = True,
                          conventions: int = 0, stream=None):
    """Recurrent path with compact capture.  Returns (out, final_state,
    state_update).  final_state may be initial_state itself (in place)."""
    T, Hk, dk, Hv, dv = _dims(q, v, B, T, cu_seqlens)
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if final_state is None and want_final_state:
        final_state = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    cap = int(state_update_capacity)
    if cap > 0 and state_update is None:
        state_update = _empty((B, cap, slot_width(Hk, Hv, dk, dv)), torch.float32, v.device,
                              stream)
    n0 = initial_state.shape[0] if initial_state is not None else 0
    st = lib().gdn_recurrent_capture(
        _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), _p(initial_state),
        _p(initial_state_indices), n0, _p(final_state), _p(out), B, T, Hk, Hk, Hv,
        dk, dv, scale, *_codes(q, alpha, conventions), cap, _p(capture_count),
        _p(state_update_active), _p(state_update), _stream(stream))
    _check(st, "gdn_recurrent_capture")
    return out, final_state, state_update


def gdn_replay_state_updates(state_in, state_update, accepted_count, *,
                             state_update_capacity: int, Hk: int,
                             state_out=None, stream=None):
    """Replay the first accepted_count[b] captured slots onto state_in.
    Returns state_out (state_in itself is allowed, in place)."""
    B, Hv, dv, dk = state_in.shape
    if state_out is None:
        state_out = _empty(state_in.shape, state_in.dtype, state_in.device, stream)
    st = lib().gdn_replay_state_updates(
        _p(state_in), _p(state_out), _p(state_update), int(state_update_capacity),
        _p(accepted_count), B, int(Hk), Hv, dk, dv, _stream(stream))
    _check(st, "gdn_replay_state_updates")
    return state_out


def gdn_replay_verify(q, k, v, alpha, beta, *, B: int, T: Optional[int] = None,
                      cu_seqlens=None, state_in=None, state_out=None,
                      prev_state_update=None, prev_capacity: int = 0,
                      accepted_count=None, draft_final_state=None, out=None,
                      scale: float = 1.0, state_update_capacity: int = 0,
                      capture_count=None, state_update_active=None,
                      state_update=None, want_draft_final_state: bool = False,
                      conventions: int = 0, stream=None):
    """One speculative step: replay the accepted prefix of prev_state_update
    onto state_in, write it to state_out (state_in itself allowed), then run
    the draft tokens with capture.  Returns (out, state_out, state_update,
    draft_final_state)."""
    T, Hk, dk, Hv, dv = _dims(q, v, B, T, cu_seqlens)
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if state_out is None:
        state_out = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    if draft_final_state is None and want_draft_final_state:
        draft_final_state = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    cap = int(state_update_capacity)
    if cap > 0 and state_update is None:
        state_update = _empty((B, cap, slot_width(Hk, Hv, dk, dv)), torch.float32, v.device,
                              stream)
    st = lib().gdn_replay_verify(
        _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), _p(state_in),
        _p(state_out), _p(prev_state_update), int(prev_capacity), _p(accepted_count),
        _p(draft_final_state), _p(out), B, T, Hk, Hk, Hv, dk, dv, scale,
        *_codes(q, alpha, conventions), cap, _p(capture_count),
        _p(state_update_active), _p(state_update), _stream(stream))
    _check(st, "gdn_replay_verify")
    return out, state_out, state_update, draft_final_state


def gdn_linear_prefill_workspace_size(B, T, Hk, Hv, dk, dv, dtype_qkv, varlen=False) -> int:
    return int(lib().gdn_linear_prefill_workspace_size(B, T, Hk, Hv, dk, dv,
                                                       _DT.get(dtype_qkv, dtype_qkv),
                                                       int(bool(varlen))))


def _is(t, shape, dtype) -> bool:
    """Whether a buffer is a raw pointer, or a tensor of this kind."""
    return isinstance(t, int) or (t.shape == shape and t.dtype == dtype)


def _linear_dims(q, k, v, alpha, cu_seqlens, initial_state, initial_state_indices, final_state,
                 out, B, T, conventions):
    """T, Hk, dk, Hv, dv and the number of initial states of a linear-attention call, with
    its tensors' shapes and dtypes checked: the library sees addresses only, and would read
    and write past the end of a smaller tensor.  (Each shape is asked for once, as that is
    what the checks cost.)"""
    total, Hk, dk = q_shape = q.shape
    rows, Hv, dv = v_shape = v.shape
    dtype = q.dtype
    if k.shape != q_shape or rows != total or k.dtype != dtype or v.dtype != dtype:
        raise ValueError("q and k are [total_T, Hk, dk], v [total_T, Hv, dv], of one dtype")
    if alpha.shape != ((Hv,) if conventions & GDN_ALPHA_PER_HEAD else (total, Hv)):
        raise ValueError("alpha is [Hv] with GDN_ALPHA_PER_HEAD and [total_T, Hv] without")
    if cu_seqlens is not None:
        T = total
        if not _is(cu_seqlens, (B + 1,), torch.int32):
            raise ValueError("cu_seqlens is int32 [B + 1]")
    elif T is None:
        T = total // B if B else 0
    elif B * T > total:
        raise ValueError("q, k and v hold B rows of T tokens")
    states = 0
    if initial_state is not None:
        states, *state = initial_state.shape
        if state != [Hv, dv, dk] or initial_state.dtype != torch.float32:
            raise ValueError("initial_state is float32 [states, Hv, dv, dk]")
        if initial_state_indices is not None and not _is(initial_state_indices, (B,), torch.int32):
            raise ValueError("initial_state_indices is int32 [B]")
    if final_state is not None and not _is(final_state, (B, Hv, dv, dk), torch.float32):
        raise ValueError("final_state is float32 [B, Hv, dv, dk]")
    if out is not None and not _is(out, v_shape, dtype):
        raise ValueError("out must have the shape and the dtype of v")
    return int(T), Hk, dk, Hv, dv, states


def gdn_linear_prefill(q, k, v, alpha, *, B: int, T: Optional[int] = None, cu_seqlens=None,
                       initial_state=None, initial_state_indices=None, final_state=None,
                       out=None, scale: float = 1.0, workspace=None,
                       want_final_state: bool = True, conventions: int = 0, stream=None):
    """Linear attention with a decay for each head, chunked form.  alpha is
    [total_T, Hv], or [Hv] with GDN_ALPHA_PER_HEAD in conventions.  Returns
    (out, final_state)."""
    T, Hk, dk, Hv, dv, n0 = _linear_dims(q, k, v, alpha, cu_seqlens, initial_state,
                                         initial_state_indices, final_state, out, B, T, conventions)
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if final_state is None and want_final_state:
        final_state = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    if workspace is None:
        need = lib().gdn_linear_prefill_workspace_size(B, T, Hk, Hv, dk, dv, _DT[q.dtype],
                                                       int(cu_seqlens is not None))
        if need > 0:
            workspace = _empty(need, torch.uint8, v.device, stream, scratch=True)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib().gdn_linear_prefill(
        _p(q), _p(k), _p(v), _p(alpha), _p(cu_seqlens), _p(initial_state),
        _p(initial_state_indices), n0, _p(final_state), _p(out), B, T, Hk, Hk, Hv, dk, dv,
        scale, _DT[q.dtype], _DT[alpha.dtype] | conventions, _p(workspace), ws_bytes,
        _stream(stream))
    _check(st, "gdn_linear_prefill")
    return out, final_state


def gdn_linear_recurrent(q, k, v, alpha, *, B: int, T: Optional[int] = None, cu_seqlens=None,
                         initial_state=None, initial_state_indices=None, final_state=None,
                         out=None, scale: float = 1.0, state_update_capacity: int = 0,
                         capture_count=None, state_update_active=None, state_update=None,
                         want_final_state: bool = True, conventions: int = 0, stream=None):
    """Linear attention token by token, with the compact capture (delta = v).
    Returns (out, final_state, state_update).  final_state may be
    initial_state itself (in place)."""
    T, Hk, dk, Hv, dv, n0 = _linear_dims(q, k, v, alpha, cu_seqlens, initial_state,
                                         initial_state_indices, final_state, out, B, T, conventions)
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if final_state is None and want_final_state:
        final_state = _empty((B, Hv, dv, dk), torch.float32, v.device, stream)
    cap = int(state_update_capacity)
    if cap > 0:
        slots = (B, cap, slot_width(Hk, Hv, dk, dv))
        if state_update is None:
            state_update = _empty(slots, torch.float32, v.device, stream)
        elif not _is(state_update, slots, torch.float32):
            raise ValueError("state_update is float32 [B, capacity, slot_width]")
        if capture_count is not None and not _is(capture_count, (B,), torch.int32):
            raise ValueError("capture_count is int32 [B]")
        if not (state_update_active is None or isinstance(state_update_active, int)
                or (state_update_active.dtype == torch.int32 and state_update_active.numel() >= 1)):
            raise ValueError("state_update_active is an int32 on the device")
    st = lib().gdn_linear_recurrent(
        _p(q), _p(k), _p(v), _p(alpha), _p(cu_seqlens), _p(initial_state),
        _p(initial_state_indices), n0, _p(final_state), _p(out), B, T, Hk, Hk, Hv, dk, dv,
        scale, _DT[q.dtype], _DT[alpha.dtype] | conventions, cap, _p(capture_count),
        _p(state_update_active), _p(state_update), _stream(stream))
    _check(st, "gdn_linear_recurrent")
    return out, final_state, state_update


def _rows(t, width_dims: int):
    """Pointer and row stride (elements) of a tensor whose rows (the last
    width_dims dimensions) are contiguous."""
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors")
    if t.is_contiguous():
        return t.data_ptr(), t.shape[1] * (t.shape[2] if width_dims == 2 else 1)
    want = 1
    for d in range(t.dim() - 1, t.dim() - 1 - width_dims, -1):
        if t.shape[d] != 1 and t.stride(d) != want:
            raise ValueError("the elements of a row must be contiguous")
        want *= t.shape[d]
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else want)


def gdn_gated_norm(x, z=None, weight=None, *, eps: float = 1e-6, gate: int = GDN_GATE_SILU,
                   out=None, stream=None):
    """Norm of each head of x [N, H, d], fused with its gate z: rmsnorm(x) *
    weight * act(z), or with GDN_GATE_FIRST rmsnorm(x * act(z)) * weight.  x, z
    and out may be slices of wider rows.  Without z the gate is none."""
    shape, dtype = x.shape, x.dtype
    N, H, d = shape
    if z is None:
        gate &= ~0xF
        zp, zs = None, H * d
    else:
        if z.shape != shape or z.dtype != dtype:
            raise ValueError("z must have the shape and the dtype of x")
        zp, zs = _rows(z, 2)
    wp, wt = None, GDN_F32
    if weight is not None:
        if weight.dim() != 1 or weight.shape[0] != d:
            raise ValueError("weight must have one element for each of a head")
        wp, wt = _p(weight), _DT[weight.dtype]
    if out is None:
        out = _empty(shape, dtype, x.device, stream)
        op, os_ = out.data_ptr(), H * d
    else:
        if out.shape != shape or out.dtype != dtype:
            raise ValueError("out must have the shape and the dtype of x")
        op, os_ = _rows(out, 2)
    xp, xs = _rows(x, 2)
    st = lib().gdn_gated_norm(xp, zp, wp, op, N, H, d, xs, zs, os_, eps, gate, _DT[dtype], wt,
                              _stream(stream))
    if st:
        _check(st, "gdn_gated_norm")
    return out


def gdn_residual_norm(y, residual=None, *, post_weight=None, gate=None,
                      gate_act: int = GDN_GATE_SIGMOID, res_scale: float = 1.0, pre_weight=None,
                      eps: float = 1e-6, unit_offset: bool = False, residual_out=None, out=None,
                      residual_dtype=None, stream=None):
    """From one block to the next: x' = residual + res_scale * act(gate) *
    [rmsnorm(y) * post_weight], and rmsnorm(x') * pre_weight.  y and gate are
    [N, D] (rows may be slices).  Returns (x', out); residual_out may be
    residual itself."""
    shape, dtype = y.shape, y.dtype
    N, D = shape
    flags = GDN_NORM_UNIT_OFFSET if unit_offset else 0
    xp, rdt = None, residual_dtype or dtype
    if residual is not None:
        if residual.shape != shape:
            raise ValueError("residual must have the shape of y")
        xp, rdt = _p(residual), residual.dtype
    gp, gs = None, D
    if gate is not None:
        if gate.shape != shape or gate.dtype != dtype:
            raise ValueError("gate must have the shape and the dtype of y")
        gp, gs = _rows(gate, 1)
        flags |= gate_act
    w1 = w2 = None
    wt = GDN_F32
    if post_weight is not None:
        if post_weight.dim() != 1 or post_weight.shape[0] != D:
            raise ValueError("a norm's weight must have one element for each of a row")
        w1, wt = _p(post_weight), _DT[post_weight.dtype]
    if pre_weight is not None:
        if pre_weight.dim() != 1 or pre_weight.shape[0] != D:
            raise ValueError("a norm's weight must have one element for each of a row")
        if w1 is not None and _DT[pre_weight.dtype] != wt:
            raise ValueError("the two weights must have one dtype")
        w2, wt = _p(pre_weight), _DT[pre_weight.dtype]
    if residual_out is None:
        residual_out = _empty(shape, rdt, y.device, stream)
    elif residual_out.shape != shape or residual_out.dtype != rdt:
        raise ValueError("residual_out must have the shape of y and the residual's dtype")
    if out is None:
        out = _empty(shape, dtype, y.device, stream)
    elif out.shape != shape or out.dtype != dtype:
        raise ValueError("out must have the shape and the dtype of y")
    yp, ys = _rows(y, 1)
    st = lib().gdn_residual_norm(yp, xp, gp, w1, w2, _p(residual_out), _p(out), N, D, ys, gs,
                                 res_scale, eps, flags, _DT[dtype], _DT[rdt], wt, _stream(stream))
    if st:
        _check(st, "gdn_residual_norm")
    return residual_out, out


def _positions(t, K: int):
    """Pointer and position stride (elements) of probabilities [B, K, V] whose
    rows are contiguous and evenly spaced (a slice of a padded vocabulary)."""
    if t.is_contiguous():
        return _p(t), t.shape[2]
    if not t.is_cuda:
        raise ValueError("libgdn takes device tensors")
    s0, s1, s2 = t.stride()
    if K == 1 and t.shape[0] > 1:  # (the stride of a dimension of one says nothing)
        s1 = s0
    if s2 != 1 or (t.shape[0] > 1 and s0 != K * s1):
        raise ValueError("probabilities must be contiguous rows, evenly spaced")
    return t.data_ptr(), s1


def gdn_accept_drafts(target_probs, draft_probs, draft_tokens, uniform, *, draft_count=None,
                      tokens=None, emitted_count=None, stream=None):
    """Verify drafts [B, K] against target_probs [B, K + 1, V] (draft_probs
    [B, K, V], or None for certain drafts) with uniform [B, K + 1].  Returns
    (tokens [B, K + 1], emitted_count [B]): the accepted drafts, one sampled
    token, then -1; emitted_count is the accepted_count of a replay."""
    B, K1, V = target_probs.shape
    K = K1 - 1
    dtype, i32 = target_probs.dtype, torch.int32
    if draft_tokens.shape != (B, K) or uniform.shape != (B, K1):
        raise ValueError("draft_tokens must be [B, K] and uniform [B, K + 1]")
    if draft_tokens.dtype != i32 or uniform.dtype != torch.float32:
        raise ValueError("draft_tokens are int32, uniform is float32")
    qp, qs = None, V
    if draft_probs is not None:
        if draft_probs.shape != (B, K, V) or draft_probs.dtype != dtype:
            raise ValueError("draft_probs must be [B, K, V] in target_probs' dtype")
        qp, qs = _positions(draft_probs, K)
    if draft_count is not None and (draft_count.shape != (B,) or draft_count.dtype != i32):
        raise ValueError("draft_count is int32 [B]")
    if tokens is None:
        tokens = _empty((B, K1), i32, target_probs.device, stream)
    elif tokens.shape != (B, K1) or tokens.dtype != i32:
        raise ValueError("tokens is int32 [B, K + 1]")
    if emitted_count is None:
        emitted_count = _empty((B,), i32, target_probs.device, stream)
    elif emitted_count.shape != (B,) or emitted_count.dtype != i32:
        raise ValueError("emitted_count is int32 [B]")
    pp, ps = _positions(target_probs, K1)
    st = lib().gdn_accept_drafts(pp, qp, _p(draft_tokens), _p(uniform), _p(draft_count),
                                 _p(tokens), _p(emitted_count), B, K, V, ps, qs, _DT[dtype],
                                 _stream(stream))
    if st:
        _check(st, "gdn_accept_drafts")
    return tokens, emitted_count


def _here(t) -> int:
    """Pointer of a tensor on the current device, the one that the kernels run on."""
    device = t.get_device()
    if device < 0:
        raise ValueError("libgdn takes device tensors")
    if device != _device():
        raise ValueError("the tensors must be on the current device")
    return t.data_ptr()


def _whole(t) -> Optional[int]:
    """Pointer of a contiguous tensor on the current device, or None."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libgdn takes contiguous tensors")
    return _here(t)


def _heads(t, N: int, H: int, d: int):
    """Pointer and token stride (elements) of heads [N, H, d] whose tokens are contiguous
    (slices of wider rows among them)."""
    s0, s1, s2 = t.stride()
    at = _here(t)
    if (s2 != 1 and d != 1) or (s1 != d and H != 1):
        raise ValueError("the elements of a token must be contiguous")
    return at, s0 if N > 1 else H * d


def _ints(t, shape, what: str):
    """Pointer of a contiguous int32 tensor of this shape."""
    if t.dtype != torch.int32 or t.shape != shape:
        raise ValueError(f"{what} is int32 {list(shape)}")
    return _whole(t)


def _fits(sizes: int) -> None:
    """Sizes, or'd together, that C ints hold (ctypes would hand on their lower 32 bits)."""
    if sizes > 0x7fffffff:
        raise ValueError("the sizes of a call must be below 2^31")


def _turn_args(inv_freq, positions, axes, N: int, d: int):
    """Pointers of inv_freq, positions and axes, R and A of a rotation of N tokens."""
    half = inv_freq.shape[0]
    if inv_freq.dim() != 1 or inv_freq.dtype != torch.float32 or 2 * half > d:
        raise ValueError("inv_freq is float32 [R / 2], R of at most a head's size")
    A, pp, ap = 1, None, None
    if positions is not None:
        if positions.dim() == 2:
            A = positions.shape[0]
            if A < 1:
                raise ValueError("positions is int32 [N] or [A, N], A of one at least")
            pp = _ints(positions, (A, N), "positions")
        else:
            pp = _ints(positions, (N,), "positions")
        if axes is not None:
            ap = _ints(axes, (half,), "axes")
    return _whole(inv_freq), pp, ap, 2 * half, A


def gdn_rotary(x, positions, inv_freq, *, axes=None, pairs: bool = False, inverse: bool = False,
               out=None, stream=None):
    """Rotary positions on the first R = 2 * inv_freq.numel() elements of each head
    of x [N, H, d] (rows may be slices).  positions [N], or [A, N] with axes
    [R / 2] naming each pair's axis.  pairs: elements 2 i and 2 i + 1 turn
    together, else i and i + R / 2.  inverse turns back, which is the gradient.
    out may be x."""
    shape, dtype = x.shape, x.dtype
    N, H, d = shape
    fp, pp, ap, R, A = _turn_args(inv_freq, positions, axes, N, d)
    _fits(H | d | A)
    xp, xs = _heads(x, N, H, d)
    if out is None:
        out = _empty(shape, dtype, x.device, stream)
        op, os_ = out.data_ptr(), H * d
    else:
        if out.shape != shape or out.dtype != dtype:
            raise ValueError("out must have the shape and the dtype of x")
        op, os_ = _heads(out, N, H, d)
    flags = (GDN_ROTARY_PAIRS if pairs else 0) | (GDN_ROTARY_INVERSE if inverse else 0)
    st = lib().gdn_rotary(xp, op, pp, ap, fp, N, H, d, R, A, xs, os_, flags, _DT[dtype], _stream(stream))
    if st:
        _check(st, "gdn_rotary")
    return out


def _page_args(k_pages, v_pages, page_table, kv_lens, B: int, dtype):
    """Shape, pointers and strides of a cache [num_pages, page_size, Hk, d] (any order of the
    first three dimensions in memory), with its table and its lengths."""
    pages, page_size, Hk, d = shape = k_pages.shape
    s0, s1, s2, s3 = strides = k_pages.stride()
    if v_pages.shape != shape or v_pages.stride() != strides:
        raise ValueError("k_pages and v_pages are [num_pages, page_size, Hk, d] with the same strides")
    if k_pages.dtype != dtype or v_pages.dtype != dtype:
        raise ValueError("the pages must have the dtype of the tokens")
    if s3 != 1 and d != 1:
        raise ValueError("the elements of a slot's head must be contiguous")
    if page_table.dim() != 2:
        raise ValueError("page_table is int32 [B, max_pages]")
    width = page_table.shape[1]
    return (Hk, d, _here(k_pages), _here(v_pages), _ints(page_table, (B, width), "page_table"),
            _ints(kv_lens, (B,), "kv_lens"), pages, page_size, width, s0, s1, s2)


def _row_count(total: int, B: int, T, cu_seqlens):
    """T argument and pointer of the rows of `total` tokens."""
    if cu_seqlens is not None:
        return total, _ints(cu_seqlens, (B + 1,), "cu_seqlens")
    if T is None:
        T = total // B if B else 0
    if B * T > total or T < 0:
        raise ValueError("the tensors hold B rows of T tokens")
    return T, None


def gdn_paged_append(k, v, k_pages, v_pages, page_table, kv_lens, *, B: int, T: Optional[int] = None,
                     cu_seqlens=None, q=None, q_out=None, inv_freq=None, positions=None, axes=None,
                     pairs: bool = False, stream=None):
    """New tokens' keys and values [total_T, Hk, d] into the cache's pages
    [num_pages, page_size, Hk, d], row b's at the positions that end at kv_lens[b].  With
    inv_freq the keys, and the queries q [total_T, Hq, d], are rotated on the way, by
    `positions` (see gdn_rotary; of the B * T tokens where rows are uniform) or by their
    positions in the cache.  Returns the rotated queries (q_out, which may be q), or None
    without q."""
    N, Hk, d = shape = k.shape
    dtype = k.dtype
    if v.shape != shape or v.dtype != dtype:
        raise ValueError("v must have the shape and the dtype of k")
    ph, pd, kp, vp, tp, lp, pages, size, width, s0, s1, s2 = _page_args(k_pages, v_pages, page_table, kv_lens, B, dtype)
    if ph != Hk or pd != d:
        raise ValueError("the pages must have the heads of k")
    T, cp = _row_count(N, B, T, cu_seqlens)
    fp = pp = ap = None
    R, A = 0, 1
    if inv_freq is not None:
        fp, pp, ap, R, A = _turn_args(inv_freq, positions, axes, N if cp is not None else B * T, d)
    Hq, qp, qs, op, os_ = 0, None, 0, None, 0
    if q is not None:
        n, Hq, e = q_shape = q.shape
        if n != N or e != d or q.dtype != dtype:
            raise ValueError("q is [total_T, Hq, d] in the dtype of k")
        qp, qs = _heads(q, N, Hq, d)
        if q_out is None:
            q_out = _empty(q_shape, dtype, q.device, stream)
            op, os_ = q_out.data_ptr(), Hq * d
        else:
            if q_out.shape != q_shape or q_out.dtype != dtype:
                raise ValueError("q_out must have the shape and the dtype of q")
            op, os_ = _heads(q_out, N, Hq, d)
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    _fits(N | Hq | Hk | d | A | pages | size | width)
    xk, ks = _heads(k, N, Hk, d)
    xv, vs = _heads(v, N, Hk, d)
    st = lib().gdn_paged_append(qp, xk, xv, op, kp, vp, tp, lp, cp, pp, ap, fp, B, T, Hq, Hk, d, R, A,
                                qs, ks, vs, os_, pages, size, width, s0, s1, s2,
                                GDN_ROTARY_PAIRS if pairs else 0, _DT[dtype], _stream(stream))
    if st:
        _check(st, "gdn_paged_append")
    return q_out


def gdn_paged_attention_workspace_size(B, T, Hq, Hk, d, dtype, varlen=False) -> int:
    return int(lib().gdn_paged_attention_workspace_size(B, T, Hq, Hk, d, _DT.get(dtype, dtype),
                                                        int(bool(varlen))))


def gdn_paged_attention(q, k_pages, v_pages, page_table, kv_lens, *, B: int, T: Optional[int] = None,
                        cu_seqlens=None, scale: Optional[float] = None, causal: bool = True,
                        window: int = 0, out=None, lse=None, want_lse: bool = False, workspace=None,
                        stream=None):
    """Attention of new tokens q [total_T, Hq, d] (rows may be slices) over the
    cache, row b's last one at position kv_lens[b] - 1: over the keys up to a query's own (with
    a window, the last `window` of them), or over all keys of the row without `causal`.  scale
    is d ** -0.5 by default.  Returns (out, lse); lse [total_T, Hq] (None unless wanted) is the
    log of the sum of weights.  Without `workspace` calls on the default stream use one that
    the thread keeps (up to 40 MB on a GB300), others allocate."""
    N, Hq, d = shape = q.shape
    dtype = q.dtype
    Hk, pd, kp, vp, tp, lp, pages, size, width, s0, s1, s2 = _page_args(k_pages, v_pages, page_table, kv_lens, B, dtype)
    if pd != d:
        raise ValueError("the pages must have the head size of q")
    T, cp = _row_count(N, B, T, cu_seqlens)
    _fits(N | Hq | Hk | d | pages | size | width | window)
    qp, qs = _heads(q, N, Hq, d)
    device = q.device
    if out is None:
        out = _empty(shape, dtype, device, stream)
        op = out.data_ptr()
    elif out.shape != shape or out.dtype != dtype:
        raise ValueError("out must have the shape and the dtype of q")
    else:
        op = _whole(out)
    if lse is None:
        if want_lse:
            lse = _empty((N, Hq), torch.float32, device, stream)
    elif lse.shape != (N, Hq) or lse.dtype != torch.float32:
        raise ValueError("lse is float32 [total_T, Hq]")
    L, code = lib(), _DT[dtype]
    handle = _stream(stream)
    kept = None
    if workspace is not None:
        wp, ws_bytes = _whole(workspace), workspace.numel() * workspace.element_size()
    else:
        if not handle:
            kept = _kept.__dict__.get(_device())
        if kept is not None:
            workspace, wp, ws_bytes = kept
        else:
            ws_bytes = L.gdn_paged_attention_workspace_size(B, T, Hq, Hk, d, code, cp is not None)
            wp = None
            if not 0 < ws_bytes < 1 << 62:
                pass
            elif not handle and not _stream(None):
                workspace, wp, _ = _keep(ws_bytes, device)
            else:
                workspace = _empty(ws_bytes, torch.uint8, device, stream, scratch=True)
                wp = workspace.data_ptr()
    if scale is None:
        scale = d ** -0.5
    flags = 0 if causal else GDN_ATTENTION_FULL
    lp_out = _whole(lse)
    st = L.gdn_paged_attention(qp, kp, vp, tp, lp, cp, op, lp_out, B, T, Hq, Hk, d, qs, pages, size, width,
                               s0, s1, s2, scale, window, flags, code, wp, ws_bytes, handle)
    if st == GDN_ERR_WORKSPACE and kept is not None:  # (nothing was launched: with one that is large enough)
        ws_bytes = L.gdn_paged_attention_workspace_size(B, T, Hq, Hk, d, code, cp is not None)
        if _stream(None):
            workspace = _empty(ws_bytes, torch.uint8, device, stream, scratch=True)
            wp = workspace.data_ptr()
        else:
            workspace, wp, _ = _keep(ws_bytes, device)
        st = L.gdn_paged_attention(qp, kp, vp, tp, lp, cp, op, lp_out, B, T, Hq, Hk, d, qs, pages, size, width,
                                   s0, s1, s2, scale, window, flags, code, wp, ws_bytes, handle)
    if st:
        _check(st, "gdn_paged_attention")
    return out, lse


def gdn_set_wait_limit_ns(ns: int) -> None:
    """Testing hook: limit of the kernels' waits on another warp's work, in
    nanoseconds (0 restores the 1 s default; below 1000 gives up at the first
    incomplete check)."""
    lib().gdn_set_wait_limit_ns(int(ns))


def gdn_device_errors(stream=None) -> int:
    """Synchronise the stream and return (and clear) the GDN_DEVERR_* bits."""
    flags = ctypes.c_uint32(0)
    st = lib().gdn_device_errors(_stream(stream), ctypes.byref(flags))
    if st not in (GDN_OK,):
        raise GdnError(st, "gdn_device_errors")
    return int(flags.value)


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def gdn_prefill_chunked_noalloc(q, k, v, alpha, beta, *, B: int, T: Optional[int] = None,
                                cu_seqlens=None, initial_state=None,
                                initial_state_indices=None, final_state, out,
                                chunk: int = 64, scale: float = 1.0, conventions: int = 0,
                                stream=None):
    """Chunked prefill that allocates nothing: the library's fixed device
    scratch replaces the workspace, and the caller passes `out` and
    `final_state` (None allowed for final_state only if not wanted).  For
    callers that cannot allocate device memory; see include/gdn.h for the size
    limit and the rule that calls must not overlap on the GPU."""
    L = lib()
    fn = L.gdn_prefill_chunked_noalloc
    if fn.restype is not ctypes.c_int or fn.argtypes is None:
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        fn.argtypes = [vp] * 8 + [i, vp, vp] + [i] * 8 + [f, i, i, vp]
        fn.restype = ctypes.c_int
    T, Hk, dk, Hv, dv = _dims(q, v, B, T, cu_seqlens)
    n0 = initial_state.shape[0] if initial_state is not None else 0
    st = fn(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), _p(initial_state),
            _p(initial_state_indices), n0, _p(final_state), _p(out), B, T, Hk, Hk, Hv, dk, dv,
            chunk, scale, *_codes(q, alpha, conventions), _stream(stream))
    _check(st, "gdn_prefill_chunked_noalloc")
    return out, final_state
