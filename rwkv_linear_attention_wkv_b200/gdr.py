"""Binding of the gated delta rule (include/wkv.h, wkv_gdr_*): argument marshalling only.

The tensors of a call must be on one device; the call runs there, on that device's current
stream (or the stream given), whichever device is current. What a call on a given stream makes
(results without a tensor to go to, scratch) comes from that stream's memory; tensors that the
caller made on another stream and lets go of before the call has run are the caller's to keep.

An ordinary call on the current stream goes through _binding.so (csrc/binding.cpp), which returns
NotImplemented for whatever it does not take; the functions here then check, explain and call.
They need libwkv.so alone.
"""
from __future__ import annotations

import ctypes
import warnings

import torch

from . import WkvError, _made, lib


class _NoBinding:
    """In the place of _binding.so: every call is left to the functions here."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


try:
    from . import _binding
    if getattr(_binding, "torch_version", None) != torch.__version__:
        raise ImportError("it was built for another torch")
except ImportError as e:
    warnings.warn(f"_binding.so is not used ({e}): calls of the gated delta rule and the norms take a "
                  "few microseconds longer; build it with "
                  "`python rwkv_linear_attention_wkv_b200/build.py`", RuntimeWarning)
    _binding = _NoBinding()

_F32 = torch.float32
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


class GdrProblem(ctypes.Structure):
    """wkv_gdr_problem of include/wkv.h."""
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("H", ctypes.c_int64), ("N", ctypes.c_int64), ("n_seqs", ctypes.c_int64),
                ("seq_offsets", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


# Fewer tokens than this are never walked in segments (include/wkv.h).
_SEGMENTED = 1024


def _at(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape, index):
    """Refuses t unless it is a contiguous tensor of this dtype and shape on CUDA device `index`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and \
                t.is_contiguous() and index >= 0:
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _run(fn, index, stream, *args):
    """Calls fn(*args, stream) with CUDA device `index` current."""
    if stream is not None and stream.device_index != index:
        raise ValueError(f"stream must be of cuda:{index}, like the tensors, got {stream.device}")
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != 0:
        raise WkvError(fn.__name__, rc)


def _scratch(nbytes, index, stream):
    """Uninitialised bytes for one call."""
    return _made(stream, lambda: torch.empty(nbytes, dtype=torch.uint8,
                                             device=torch.device("cuda", index)))


def _bytes(fn, problem, index):
    """A size that depends on the device."""
    if index == torch._C._cuda_getDevice():
        return int(fn(problem))
    with torch.cuda.device(index):
        return int(fn(problem))


def _shape(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.shape


def _problem(q, v, n, scale, seq_offsets=None):
    """Problem and device of a call from q (n dimensions, Hk, N) and v (n dimensions, H, N)."""
    heads, shape = _shape(q, "q"), _shape(v, "v")
    if len(heads) != n + 2 or len(shape) != n + 2:
        raise ValueError(f"q and v must have {n + 2} dimensions")
    dtype = _DTYPES.get(v.dtype)
    if dtype is None:
        raise TypeError(f"v must be torch.float32 or torch.bfloat16, got {v.dtype}")
    p = GdrProblem(shape[0], shape[1] if n == 2 else 1, heads[n], shape[n], shape[n + 1], 0, None,
                   dtype, scale, None, 0)
    index = v.get_device()
    if seq_offsets is not None:
        if len(_shape(seq_offsets, "seq_offsets")) != 1 or seq_offsets.numel() < 1:
            raise ValueError("seq_offsets must hold one offset more than there are sequences")
        _need(seq_offsets, "seq_offsets", torch.int32, seq_offsets.shape, index)
        if shape[0] != 1:
            raise ValueError("with seq_offsets the sequences are packed into one row (B = 1)")
        p.n_seqs = seq_offsets.numel() - 1
        p.seq_offsets = seq_offsets.data_ptr()
    return p, index


def _inputs(q, k, v, g, beta, index):
    dt, wide = v.dtype, v.shape
    heads, qk = wide[:-1], q.shape
    _need(v, "v", dt, wide, index)
    _need(q, "q", dt, wide[:-2] + (qk[-2], wide[-1]), index)
    _need(k, "k", dt, qk, index)
    _need(g, "g", _F32, heads, index)
    _need(beta, "beta", _F32, heads, index)


def _forward(q, k, v, g, beta, state, scale, seq_offsets, y, state_out, want_state, stream):
    """Problem, outputs, device and scratch (to be held until the call is made) of a forward."""
    p, index = _problem(q, v, 2, scale, seq_offsets)
    _inputs(q, k, v, g, beta, index)
    if y is None:
        y = _made(stream, lambda: torch.empty_like(v))
    else:
        _need(y, "y", v.dtype, v.shape, index)
    B, T, H, N = v.shape
    states = (B if seq_offsets is None else p.n_seqs, H, N, N)
    if state is not None:
        _need(state, "state", _F32, states, index)
    if not want_state:
        state_out = None
    elif state_out is None:
        state_out = _made(stream, lambda: v.new_empty(states, dtype=_F32))
    else:
        _need(state_out, "state_out", _F32, states, index)
    scratch = None
    if T >= _SEGMENTED:
        nbytes = _bytes(lib.wkv_gdr_forward_workspace_bytes, ctypes.byref(p), index)
        if nbytes:
            scratch = _scratch(nbytes, index, stream)
            p.workspace, p.workspace_bytes = scratch.data_ptr(), nbytes
    return p, y, state_out, index, scratch


def wkv_gdr_forward(q, k, v, g, beta, state=None, scale=1.0, seq_offsets=None, y=None,
                    state_out=None, want_state=True, stream=None):
    """Gated delta rule per head: q, k (B, T, Hk, N); v (B, T, H, N), bf16 or fp32; g
    (log-decay) and beta (write strength) fp32 (B, T, H); N = 64 or 128, Hk divides H.

    seq_offsets (int32, n + 1) packs n sequences into one row (B = 1). state: (sequences, H,
    N, N) fp32 or None (zero). Returns (y, S_T), or (y, None) with want_state=False. state_out
    may be `state` itself. Rows of y that no packed sequence covers are left as they were
    (uninitialised without `y`).
    """
    if stream is None:
        done = _binding.gdr_forward(q, k, v, g, beta, state, scale, seq_offsets, y, state_out,
                                    want_state)
        if done is not NotImplemented:
            return done
    p, y, s1, index, _held = _forward(q, k, v, g, beta, state, scale, seq_offsets, y, state_out,
                                      want_state, stream)
    _run(lib.wkv_gdr_forward, index, stream, ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         g.data_ptr(), beta.data_ptr(), y.data_ptr(), _at(state), _at(s1))
    return y, s1


def _buffer(t, name, nbytes, index, stream):
    if t is None:
        return _scratch(nbytes, index, stream)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index or not t.is_contiguous() or \
            t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} must be a contiguous CUDA tensor of at least {nbytes} bytes on "
                         f"cuda:{index}")
    return t


def wkv_gdr_forward_checkpointed(q, k, v, g, beta, state=None, scale=1.0, seq_offsets=None, y=None,
                                 state_out=None, want_state=True, workspace=None, stream=None):
    """wkv_gdr_forward that also keeps what wkv_gdr_backward reads. Returns (y, S_T, workspace);
    hand the workspace (it is only read there) to the backward of the same inputs. seq_offsets
    must not decrease. state_out must not be `state` if `state` is needed again."""
    if stream is None:
        done = _binding.gdr_forward_checkpointed(q, k, v, g, beta, state, scale, seq_offsets, y,
                                                 state_out, want_state, workspace)
        if done is not NotImplemented:
            return done
    p, y, s1, index, _held = _forward(q, k, v, g, beta, state, scale, seq_offsets, y, state_out,
                                      want_state, stream)
    nbytes = int(lib.wkv_gdr_checkpoint_bytes(ctypes.byref(p)))
    workspace = _buffer(workspace, "workspace", nbytes, index, stream)
    _run(lib.wkv_gdr_forward_checkpointed, index, stream, ctypes.byref(p), q.data_ptr(), k.data_ptr(),
         v.data_ptr(), g.data_ptr(), beta.data_ptr(), y.data_ptr(), _at(state), _at(s1),
         _at(workspace), workspace.numel() * workspace.element_size())
    return y, s1, workspace


def wkv_gdr_backward(q, k, v, g, beta, dy, workspace, grad_state=None, scale=1.0, seq_offsets=None,
                     want_dstate=True, grads=None, scratch=None, stream=None):
    """Gradients of sum(dy * y) + sum(grad_state * S_T) for wkv_gdr_forward_checkpointed's call
    with the same inputs, whose workspace this takes. Returns a dict of dq, dk, dv (as q, k, v),
    dg, dbeta (fp32) and dstate (fp32; None with want_dstate=False).

    grads: such a dict to write into. Rows of the gradients that no packed sequence covers are
    left as they were (uninitialised without `grads`)."""
    if stream is None and grads is None and scratch is None:
        done = _binding.gdr_backward(q, k, v, g, beta, dy, workspace, grad_state, scale,
                                     seq_offsets, want_dstate)
        if done is not NotImplemented:
            return done
    p, index = _problem(q, v, 2, scale, seq_offsets)
    _inputs(q, k, v, g, beta, index)
    _need(dy, "dy", v.dtype, v.shape, index)
    B, T, H, N = v.shape
    states = (B if seq_offsets is None else p.n_seqs, H, N, N)
    if grad_state is not None:
        _need(grad_state, "grad_state", _F32, states, index)
    if grads is None:
        grads = {n: _made(stream, lambda: torch.empty_like(t)) for n, t in
                 (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
        if want_dstate:
            grads["dstate"] = _made(stream, lambda: v.new_empty(states, dtype=_F32))
    else:
        for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
            _need(grads.get(n), n, t.dtype, t.shape, index)
        if want_dstate:
            _need(grads.get("dstate"), "dstate", _F32, states, index)
    problem = ctypes.byref(p)
    nbytes = int(lib.wkv_gdr_checkpoint_bytes(problem))
    if workspace is None:
        raise TypeError("workspace must be the forward's")
    _buffer(workspace, "workspace", nbytes, index, stream)
    if scratch is None:
        nbytes = _bytes(lib.wkv_gdr_backward_workspace_bytes, problem, index)
    scratch = _buffer(scratch, "scratch", nbytes, index, stream)
    _run(lib.wkv_gdr_backward, index, stream, problem, q.data_ptr(), k.data_ptr(), v.data_ptr(),
         g.data_ptr(), beta.data_ptr(), dy.data_ptr(), workspace.data_ptr(),
         workspace.numel() * workspace.element_size(), _at(grad_state),
         *[grads[n].data_ptr() for n in ("dq", "dk", "dv", "dg", "dbeta")],
         grads["dstate"].data_ptr() if want_dstate else None, scratch.data_ptr(),
         scratch.numel() * scratch.element_size())
    return {n: grads[n] if n != "dstate" or want_dstate else None
            for n in ("dq", "dk", "dv", "dg", "dbeta", "dstate")}


def wkv_gdr_decode_step(q, k, v, g, beta, state, slots=None, scale=1.0, y=None, stream=None):
    """One token of n rows: q, k (n, Hk, N); v (n, H, N), bf16 or fp32; g, beta fp32 (n, H).

    state: (slots, H, N, N) fp32, updated in place; slots: int32 (n,), the state of each row
    (no slot twice; outside [0, len(state)): padding, the row is skipped and its y stays as it
    was, uninitialised without `y`), None = row i has state i. Returns y (n, H, N).
    """
    if stream is None:
        done = _binding.gdr_decode(q, k, v, g, beta, state, slots, scale, y)
        if done is not NotImplemented:
            return done
    p, index = _problem(q, v, 1, scale)
    _inputs(q, k, v, g, beta, index)
    n, H, N = v.shape
    pool = _shape(state, "state")
    if len(pool) != 4:
        raise ValueError("state must be (slots, H, N, N)")
    n_slots = pool[0]
    _need(state, "state", _F32, (n_slots, H, N, N), index)
    if slots is not None:
        _need(slots, "slots", torch.int32, (n,), index)
    elif n_slots < n:
        raise ValueError(f"state must have at least {n} slots, got {n_slots}")
    if y is None:
        y = _made(stream, lambda: torch.empty_like(v))
    else:
        _need(y, "y", v.dtype, v.shape, index)
    _run(lib.wkv_gdr_decode_step, index, stream, ctypes.byref(p), q.data_ptr(), k.data_ptr(),
         v.data_ptr(), g.data_ptr(), beta.data_ptr(), y.data_ptr(), state.data_ptr(), n_slots,
         _at(slots))
    return y
