"""The library's operators as PyTorch autograd functions (argument marshalling only).

The news page "RWKV CUDA linear attention GPU" describes the CUDA operator being used
from PyTorch through an autograd function whose forward and backward are fused kernels.
This module is that wrapper over the library's C ABI: the forward is
`wkv_forward_checkpointed` (y, and the state entering every 16-token chunk kept in a
workspace saved for the backward), the backward is `wkv_backward_checkpointed` (dk, dv,
dr, dw, du from those checkpoints). Nothing here computes: every number comes from the
library's kernels, on the current CUDA stream, in fp32.

    y = wkv(w, u, k, v, r)        # w, u: (C,) fp32, w > 0; k, v, r: (B, T, C) fp32 CUDA
    (y * dy).sum().backward()     # gradients for w, u, k, v and r

w is the positive decay itself (the per-token factor is e^{-w}), so w's gradient is with
respect to w, not log w. r may be None (no gate).

`gated_delta_rule` and `norm_gate` are the matrix-state update with a decay and a write strength
per token, and the norms, gate and residual around a block, in the same manner (bf16 or fp32).
"""
import torch
from torch.autograd.function import once_differentiable

from . import (wkv_backward_checkpointed, wkv_forward_checkpointed, wkv_gdr_backward,
               wkv_gdr_forward, wkv_gdr_forward_checkpointed, wkv_norm_gate_backward,
               wkv_norm_gate_forward)


class WKVFunction(torch.autograd.Function):
    """y = sigmoid(r) * wkv(w, u, k, v) with its gradients from the library's kernels."""

    @staticmethod
    def forward(ctx, w, u, k, v, r):
        w, u, k, v = (t.contiguous() for t in (w, u, k, v))
        r = None if r is None else r.contiguous()
        y, workspace = wkv_forward_checkpointed(w, u, k, v, r)
        ctx.save_for_backward(w, u, k, v, r, workspace)
        ctx.has_r = r is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        w, u, k, v, r, workspace = ctx.saved_tensors
        g = wkv_backward_checkpointed(w, u, k, v, r if ctx.has_r else None, dy.contiguous(),
                                      workspace, want_dr=ctx.has_r)
        return g["dw"], g["du"], g["dk"], g["dv"], g["dr"]


def wkv(w, u, k, v, r=None):
    """Differentiable WKV: see WKVFunction."""
    return WKVFunction.apply(w, u, k, v, r)


def _dense(t):
    """t as the rule's kernels read it: contiguous, at a multiple of 16 bytes. A view or a gradient
    may be contiguous and start anywhere."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _read_outs(v, seq_offsets):
    # tokens that no packed sequence covers are not written
    return torch.empty_like(v) if seq_offsets is None else torch.zeros_like(v)


class GatedDeltaRuleFunction(torch.autograd.Function):
    """(y, final states) of the gated delta rule with the library's gradients for q, k, v, g, beta
    and the initial states."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, state, scale, seq_offsets):
        q, k, v, g, beta, state = map(_dense, (q, k, v, g, beta, state))
        y = _read_outs(v, seq_offsets)
        y, last, workspace = wkv_gdr_forward_checkpointed(q, k, v, g, beta, state=state, scale=scale,
                                                          seq_offsets=seq_offsets, y=y)
        ctx.save_for_backward(q, k, v, g, beta, seq_offsets, workspace)
        ctx.scale, ctx.has_state = scale, state is not None
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        if dy is None and dlast is None:
            return (None,) * 8
        q, k, v, g, beta, seq_offsets, workspace = ctx.saved_tensors
        dy = torch.zeros_like(v) if dy is None else _dense(dy)
        dlast = _dense(dlast)
        grads = None
        if seq_offsets is not None:
            grads = {"d" + n: torch.zeros_like(t) for n, t in
                     (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta))}
            if ctx.has_state:
                H, N = v.shape[2:]
                grads["dstate"] = v.new_empty(seq_offsets.numel() - 1, H, N, N, dtype=torch.float32)
        d = wkv_gdr_backward(q, k, v, g, beta, dy, workspace, grad_state=dlast, scale=ctx.scale,
                             seq_offsets=seq_offsets, want_dstate=ctx.has_state, grads=grads)
        return d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"], d["dstate"], None, None


def gated_delta_rule(q, k, v, g, beta, state=None, scale=1.0, seq_offsets=None):
    """Differentiable wkv_gdr_forward: (y, final states), with gradients for q, k, v, g, beta and
    state, through both results. With seq_offsets, y and the gradients are zero at tokens that no
    sequence covers. Types and shapes as wkv_gdr_forward; inputs may be non-contiguous and start
    at any element."""
    inputs = (q, k, v, g, beta, state)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        return GatedDeltaRuleFunction.apply(*inputs, scale, seq_offsets)
    # nothing to keep for a backward (every token's error and the chunks' states: more than the inputs)
    q, k, v, g, beta, state = map(_dense, inputs)
    return wkv_gdr_forward(q, k, v, g, beta, state=state, scale=scale, seq_offsets=seq_offsets,
                           y=_read_outs(v, seq_offsets))


class NormGateFunction(torch.autograd.Function):
    """(out, y) of wkv_norm_gate_forward with the library's gradients."""

    @staticmethod
    def forward(ctx, h, weight, gate, x, scale, next_weight, group, act, eps):
        h, weight, gate, x, scale, next_weight = (
            None if t is None else t.contiguous() for t in (h, weight, gate, x, scale, next_weight))
        out, y = wkv_norm_gate_forward(h, weight, gate=gate, x=x, scale=scale,
                                       next_weight=next_weight, group=group, act=act, eps=eps)
        ctx.save_for_backward(h, weight, gate, x, scale, next_weight)
        ctx.how = dict(group=group, act=act, eps=eps)
        ctx.set_materialize_grads(False)
        return out, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dy):
        if dout is None and dy is None:
            return (None,) * 9
        h, weight, gate, x, scale, next_weight = ctx.saved_tensors
        g = wkv_norm_gate_backward(h, weight, None if dout is None else dout.contiguous(), gate=gate,
                                   x=x, scale=scale, next_weight=next_weight,
                                   dy=None if dy is None else dy.contiguous(), **ctx.how)
        return (g["dh"], g["dweight"], g["dgate"], g["dx"], g["dscale"], g["dnext_weight"], None,
                None, None)


def norm_gate(h, weight=None, gate=None, x=None, scale=None, next_weight=None, group=None,
              act="silu", eps=1e-6):
    """Differentiable wkv_norm_gate_forward: (out, y), y None without next_weight."""
    return NormGateFunction.apply(h, weight, gate, x, scale, next_weight, group, act, eps)
