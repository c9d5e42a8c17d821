"""Binding of the norms around a block (include/wkv.h, wkv_norm_gate_*): argument marshalling only.

As in gdr.py, the tensors of a call must be on one device, and the call runs there; ordinary calls
go through _binding.so.
"""
from __future__ import annotations

import ctypes

import torch

from . import _made, lib
from .gdr import _binding, _DTYPES, _F32, _at, _buffer, _need, _run

_ACTS = {"none": 0, "sigmoid": 1, "silu": 2}


class NormGateProblem(ctypes.Structure):
    """wkv_norm_gate_problem of include/wkv.h."""
    _fields_ = [("R", ctypes.c_int64), ("C", ctypes.c_int64), ("group", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("act", ctypes.c_int), ("eps", ctypes.c_float)]


def _problem(h, weight, gate, x, scale, next_weight, group, act, eps):
    if not isinstance(h, torch.Tensor):
        raise TypeError("h must be a torch.Tensor")
    if h.dim() < 1:
        raise ValueError("h must be (..., C)")
    if h.dtype not in _DTYPES:
        raise TypeError(f"h must be torch.float32 or torch.bfloat16, got {h.dtype}")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {tuple(_ACTS)}, got {act!r}")
    if (gate is None) != (act == "none"):
        raise ValueError("act must be 'none' without a gate, and not with one")
    if scale is not None and x is None:
        raise ValueError("scale is the residual's: it needs x")
    shape, dt, index = h.shape, h.dtype, h.get_device()
    C = shape[-1]
    group = C if group is None else group
    if C and (group <= 0 or C % group):
        raise ValueError(f"group must divide C = {C}, got {group}")
    _need(h, "h", dt, shape, index)
    for n, t in (("gate", gate), ("x", x)):
        if t is not None:
            _need(t, n, dt, shape, index)
    for n, t in (("weight", weight), ("scale", scale), ("next_weight", next_weight)):
        if t is not None:
            _need(t, n, _F32, (C,), index)
    return (NormGateProblem(h.numel() // C if C else 0, C, group, _DTYPES[dt], _ACTS[act], eps),
            index)


def wkv_norm_gate_forward(h, weight=None, gate=None, x=None, scale=None, next_weight=None,
                          group=None, act="silu", eps=1e-6, out=None, y=None, stream=None):
    """out = x + scale * act(gate) * weight * h / RMS(h over groups of `group` channels) and, with
    next_weight, y = next_weight * out / RMS(out). h, gate, x: (..., C) bf16 or fp32; weight,
    scale, next_weight: fp32 (C,). gate (with act="none"), weight, x, scale and next_weight may
    be left out. group: default C. Returns (out, y), y None without next_weight; `out` may be h
    or x itself."""
    if stream is None:
        done = _binding.norm_gate_forward(h, weight, gate, x, scale, next_weight, group, act, eps,
                                          out, y)
        if done is not NotImplemented:
            return done
    p, index = _problem(h, weight, gate, x, scale, next_weight, group, act, eps)
    dt = h.dtype
    if out is None:
        out = _made(stream, lambda: torch.empty_like(h))
    else:
        _need(out, "out", dt, h.shape, index)
    if next_weight is None:
        if y is not None:
            raise ValueError("y needs next_weight")
    elif y is None:
        y = _made(stream, lambda: torch.empty_like(h))
    else:
        _need(y, "y", dt, h.shape, index)
    _run(lib.wkv_norm_gate_forward, index, stream, ctypes.byref(p), h.data_ptr(), _at(weight), _at(gate),
         _at(x), _at(scale), _at(next_weight), out.data_ptr(), _at(y))
    return out, y


def wkv_norm_gate_workspace_bytes(R: int, C: int) -> int:
    return int(lib.wkv_norm_gate_workspace_bytes(R, C))


def wkv_norm_gate_backward(h, weight, dout, gate=None, x=None, scale=None, next_weight=None, dy=None,
                           group=None, act="silu", eps=1e-6, workspace=None, stream=None):
    """Gradients of sum(dout * out) + sum(dy * y) for wkv_norm_gate_forward's (out, y). dout or dy
    may be None (zero). Returns a dict of dh, dgate, dx (as h) and dweight, dscale, dnext_weight
    (fp32), None where the forward had no such input (dnext_weight also without dy)."""
    if stream is None and workspace is None:
        done = _binding.norm_gate_backward(h, weight, dout, gate, x, scale, next_weight, dy, group,
                                           act, eps)
        if done is not NotImplemented:
            return done
    if dout is None and dy is None:
        raise ValueError("dout or dy must be given")
    if dy is not None and next_weight is None:
        raise ValueError("dy needs next_weight")
    p, index = _problem(h, weight, gate, x, scale, next_weight, group, act, eps)
    dt = h.dtype
    for n, t in (("dout", dout), ("dy", dy)):
        if t is not None:
            _need(t, n, dt, h.shape, index)
    like = lambda t: None if t is None else _made(stream, lambda: torch.empty_like(t))  # noqa: E731
    g = {"dh": like(h), "dweight": like(weight), "dgate": like(gate), "dx": like(x),
         "dscale": like(scale), "dnext_weight": None if dy is None else like(next_weight)}
    workspace = _buffer(workspace, "workspace", wkv_norm_gate_workspace_bytes(p.R, p.C), index,
                        stream)
    _run(lib.wkv_norm_gate_backward, index, stream, ctypes.byref(p), h.data_ptr(), _at(weight), _at(gate),
         _at(x), _at(scale), _at(next_weight), _at(dout), _at(dy), g["dh"].data_ptr(),
         _at(g["dweight"]), _at(g["dgate"]), _at(g["dx"]), _at(g["dscale"]), _at(g["dnext_weight"]),
         workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return g
