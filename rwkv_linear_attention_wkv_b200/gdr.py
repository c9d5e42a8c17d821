"""Binding of the gated delta rule (include/wkv.h, wkv_gdr_*): argument marshalling only.

The tensors of a call must be on one device; the call runs there, on that device's current
stream (or the stream given), whichever device is current.
"""
from __future__ import annotations

import ctypes

import torch

from . import WkvError, _dims, lib

_F32 = torch.float32
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


class GdrProblem(ctypes.Structure):
    """wkv_gdr_problem of include/wkv.h."""
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("H", ctypes.c_int64), ("N", ctypes.c_int64), ("n_seqs", ctypes.c_int64),
                ("seq_offsets", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float)]


def _at(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape, device):
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
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _run(fn, device, stream, *args):
    """Calls fn(*args, stream) with `device` current."""
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        rc = getattr(lib, fn)(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = getattr(lib, fn)(*args, raw)
    if rc != 0:
        raise WkvError(fn, rc)


def _problem(q, v, lead, scale, seq_offsets=None):
    """Dtype, device and problem of a call from q (*lead, Hk, N) and v (*lead, H, N)."""
    n = len(lead)
    if not _dims(q, "q", n + 2) or not _dims(v, "v", n + 2):
        raise ValueError(f"q and v must have {n + 2} dimensions")
    if v.dtype not in _DTYPES:
        raise TypeError(f"v must be torch.float32 or torch.bfloat16, got {v.dtype}")
    shape = v.shape
    p = GdrProblem(shape[0], shape[1] if n == 2 else 1, q.shape[n], shape[n], shape[n + 1], 0, None,
                   _DTYPES[v.dtype], scale)
    if seq_offsets is not None:
        if not _dims(seq_offsets, "seq_offsets", 1) or seq_offsets.numel() < 1:
            raise ValueError("seq_offsets must hold one offset more than there are sequences")
        _need(seq_offsets, "seq_offsets", torch.int32, seq_offsets.shape, v.device)
        if shape[0] != 1:
            raise ValueError("with seq_offsets the sequences are packed into one row (B = 1)")
        p.n_seqs = seq_offsets.numel() - 1
        p.seq_offsets = seq_offsets.data_ptr()
    return p


def _inputs(q, k, v, g, beta, lead):
    dt, dev = v.dtype, v.device
    qk, heads = q.shape, v.shape[:-1]
    _need(v, "v", dt, v.shape, dev)
    _need(q, "q", dt, lead + (qk[-2], v.shape[-1]), dev)
    _need(k, "k", dt, qk, dev)
    _need(g, "g", _F32, heads, dev)
    _need(beta, "beta", _F32, heads, dev)


def _sequences(p):
    return p.n_seqs if p.seq_offsets else p.B


def _forward(q, k, v, g, beta, state, scale, seq_offsets, y, state_out, want_state):
    p = _problem(q, v, (0, 0), scale, seq_offsets)
    _inputs(q, k, v, g, beta, v.shape[:2])
    dev = v.device
    if y is None:
        y = torch.empty_like(v)
    else:
        _need(y, "y", v.dtype, v.shape, dev)
    states = (_sequences(p), p.H, p.N, p.N)
    if state is not None:
        _need(state, "state", _F32, states, dev)
    s1 = None
    if want_state:
        s1 = torch.empty(states, dtype=_F32, device=dev) if state_out is None else state_out
        _need(s1, "state_out", _F32, states, dev)
    return p, y, s1, dev


def wkv_gdr_forward(q, k, v, g, beta, state=None, scale=1.0, seq_offsets=None, y=None,
                    state_out=None, want_state=True, stream=None):
    """Gated delta rule per head: q, k (B, T, Hk, N); v (B, T, H, N), bf16 or fp32; g
    (log-decay) and beta (write strength) fp32 (B, T, H); N = 64 or 128, Hk divides H.

    seq_offsets (int32, n + 1) packs n sequences into one row (B = 1). state: (sequences, H,
    N, N) fp32 or None (zero). Returns (y, S_T), or (y, None) with want_state=False. state_out
    may be `state` itself.
    """
    p, y, s1, dev = _forward(q, k, v, g, beta, state, scale, seq_offsets, y, state_out, want_state)
    _run("wkv_gdr_forward", dev, stream, ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         g.data_ptr(), beta.data_ptr(), y.data_ptr(), _at(state), _at(s1))
    return y, s1


def _buffer(t, name, nbytes, device):
    if t is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.device != device or not t.is_contiguous() or \
            t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} must be a contiguous CUDA tensor of at least {nbytes} bytes on "
                         f"{device}")
    return t


def wkv_gdr_forward_checkpointed(q, k, v, g, beta, state=None, scale=1.0, seq_offsets=None, y=None,
                                 state_out=None, want_state=True, workspace=None, stream=None):
    """wkv_gdr_forward that also keeps what wkv_gdr_backward reads. Returns (y, S_T, workspace);
    hand the workspace (it is only read there) to the backward of the same inputs. seq_offsets
    must not decrease. state_out must not be `state` if `state` is needed again."""
    p, y, s1, dev = _forward(q, k, v, g, beta, state, scale, seq_offsets, y, state_out, want_state)
    nbytes = int(lib.wkv_gdr_checkpoint_bytes(ctypes.byref(p)))
    workspace = _buffer(workspace, "workspace", nbytes, dev)
    _run("wkv_gdr_forward_checkpointed", dev, stream, ctypes.byref(p), q.data_ptr(), k.data_ptr(),
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
    p = _problem(q, v, (0, 0), scale, seq_offsets)
    _inputs(q, k, v, g, beta, v.shape[:2])
    dev = v.device
    _need(dy, "dy", v.dtype, v.shape, dev)
    states = torch.Size((_sequences(p), p.H, p.N, p.N))
    if grad_state is not None:
        _need(grad_state, "grad_state", _F32, states, dev)
    shapes = {"dq": (q.dtype, q.shape), "dk": (q.dtype, q.shape), "dv": (v.dtype, v.shape),
              "dg": (_F32, g.shape), "dbeta": (_F32, g.shape)}
    if want_dstate:
        shapes["dstate"] = (_F32, states)
    if grads is None:
        grads = {n: torch.empty(s, dtype=t, device=dev) for n, (t, s) in shapes.items()}
    else:
        for n, (t, s) in shapes.items():
            _need(grads.get(n), n, t, s, dev)
    nbytes = int(lib.wkv_gdr_checkpoint_bytes(ctypes.byref(p)))
    if workspace is None:
        raise TypeError("workspace must be the forward's")
    _buffer(workspace, "workspace", nbytes, dev)
    scratch = _buffer(scratch, "scratch",
                      int(lib.wkv_gdr_backward_workspace_bytes(ctypes.byref(p))), dev)
    _run("wkv_gdr_backward", dev, stream, ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         g.data_ptr(), beta.data_ptr(), dy.data_ptr(), _at(workspace), workspace.numel() * workspace.element_size(),
         _at(grad_state), *[grads[n].data_ptr() for n in ("dq", "dk", "dv", "dg", "dbeta")],
         _at(grads["dstate"]) if want_dstate else None, _at(scratch),
         scratch.numel() * scratch.element_size())
    return {n: grads.get(n) if n in shapes else None
            for n in ("dq", "dk", "dv", "dg", "dbeta", "dstate")}


def wkv_gdr_decode_step(q, k, v, g, beta, state, slots=None, scale=1.0, y=None, stream=None):
    """One token of n rows: q, k (n, Hk, N); v (n, H, N), bf16 or fp32; g, beta fp32 (n, H).

    state: (slots, H, N, N) fp32, updated in place; slots: int32 (n,), the state of each row
    (no slot twice; outside [0, len(state)): padding, the row is skipped and its y stays as it
    was), None = row i has state i. Returns y (n, H, N).
    """
    p = _problem(q, v, (0,), scale)
    _inputs(q, k, v, g, beta, v.shape[:1])
    dev = v.device
    if not _dims(state, "state", 4):
        raise ValueError("state must be (slots, H, N, N)")
    n_slots = state.shape[0]
    _need(state, "state", _F32, (n_slots, p.H, p.N, p.N), dev)
    if slots is not None:
        _need(slots, "slots", torch.int32, (p.B,), dev)
    elif n_slots < p.B:
        raise ValueError(f"state must have at least {p.B} slots, got {n_slots}")
    if y is None:
        y = torch.empty_like(v)
    else:
        _need(y, "y", v.dtype, v.shape, dev)
    _run("wkv_gdr_decode_step", dev, stream, ctypes.byref(p), q.data_ptr(), k.data_ptr(),
         v.data_ptr(), g.data_ptr(), beta.data_ptr(), y.data_ptr(), state.data_ptr(), n_slots,
         _at(slots))
    return y
