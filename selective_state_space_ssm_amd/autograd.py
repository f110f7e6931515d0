"""torch.autograd wrappers over the C ABI: the forward keeps only the chunk
states (ssm_scan_fwd_states / ssm_scan_fwd_conv with ``state_chunk``), the
backward recomputes from them (ssm_scan_bwd / ssm_scan_bwd_conv).  Argument
marshalling only; every step runs in the library's kernels.

    y, last_state = selective_scan(u, delta, A, B, C, D, z, delta_bias,
                                   delta_softplus=True, h0=None, state_chunk=128)
    y, last_state = selective_scan_conv(x, conv_w, conv_b, delta, A, B, C, D, z, ...)
    out = out_proj(y, W)          # the Linear after the gate, [b, L, d_model]
    o, last_state = head_scan(q, k, v, g=g)   # one decay per head, matrix state
    o, last_state = delta_scan(q, k, v, beta, g=g)   # the same with the gated delta rule
    y = gate_norm(x, weight, z, groups=heads)   # grouped norm of token rows with a SiLU gate
    y, h = add_norm(x, residual, weight)   # h = x + residual, its root-mean-square norm
    out = linear(y, W, bias, residual, act="silu")   # act(y W^T + bias) + residual

Gradients flow to every tensor argument that requires them (dB and dC are
computed in float32 and returned in the dtype of B and C).

A backward pass may be captured into a HIP graph.  torch's own rule for it:
no graph of the same leaves that was recorded outside the capture may still be
alive then (its accumulation nodes belong to the other stream, and waiting for
them ends the capture and the process); drop such outputs first.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (ssm_add_norm, ssm_add_norm_bwd, ssm_delta_scan_bwd, ssm_delta_scan_fwd, ssm_gate_norm,
               ssm_gate_norm_bwd, ssm_head_scan_bwd, ssm_head_scan_fwd, ssm_linear, ssm_linear_bwd, ssm_out_proj,
               ssm_out_proj_bwd, ssm_scan_bwd, ssm_scan_bwd_conv,
               ssm_scan_fwd_conv, ssm_scan_fwd_states)

__all__ = ["selective_scan", "selective_scan_conv", "out_proj", "head_scan", "delta_scan", "gate_norm", "add_norm",
           "linear"]


def _grad_or_zero(g, like):
    return torch.zeros_like(like) if g is None else g.contiguous()


def _dense(g):
    """A gradient as the library takes it: contiguous and 16-byte aligned (that of a concatenation is a view of any
    alignment)."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, h0, delta_softplus, state_chunk):
        y, last, cs = ssm_scan_fwd_states(u, delta, A, B, C, D, z, delta_bias, delta_softplus=delta_softplus,
                                          h0=h0, state_chunk=state_chunk)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, h0, cs)
        ctx.delta_softplus = delta_softplus
        ctx.state_chunk = state_chunk
        return y, last

    @staticmethod
    def backward(ctx, dy, dlast):
        u, delta, A, B, C, D, z, delta_bias, h0, cs = ctx.saved_tensors
        g = ssm_scan_bwd(u, delta, A, B, C, cs, ctx.state_chunk, _grad_or_zero(dy, u), D=D, z=z,
                         delta_bias=delta_bias, delta_softplus=ctx.delta_softplus, h0=h0,
                         dlast=None if dlast is None else dlast.contiguous(),
                         want_dD=D is not None, want_ddelta_bias=delta_bias is not None, want_dh0=h0 is not None)
        return (g["du"], g["ddelta"], g["dA"], g["dB"].to(B.dtype), g["dC"].to(C.dtype), g["dD"], g["dz"],
                g["ddelta_bias"], g["dh0"], None, None)


def selective_scan(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                   h0: Optional[torch.Tensor] = None, state_chunk: int = 128):
    """Differentiable selective scan: returns (y, last_state)."""
    return _SelectiveScan.apply(u, delta, A, B, C, D, z, delta_bias, h0, delta_softplus, state_chunk)


class _SelectiveScanConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, conv_w, conv_b, delta, A, B, C, D, z, delta_bias, h0, delta_softplus, state_chunk):
        y, last, cs, _ = ssm_scan_fwd_conv(x, conv_w, delta, A, B, C, conv_b=conv_b, D=D, z=z,
                                           delta_bias=delta_bias, delta_softplus=delta_softplus, h0=h0,
                                           state_chunk=state_chunk)
        ctx.save_for_backward(x, conv_w, conv_b, delta, A, B, C, D, z, delta_bias, h0, cs)
        ctx.delta_softplus = delta_softplus
        ctx.state_chunk = state_chunk
        return y, last

    @staticmethod
    def backward(ctx, dy, dlast):
        x, conv_w, conv_b, delta, A, B, C, D, z, delta_bias, h0, cs = ctx.saved_tensors
        g = ssm_scan_bwd_conv(x, conv_w, delta, A, B, C, cs, ctx.state_chunk, _grad_or_zero(dy, x), conv_b=conv_b,
                              D=D, z=z, delta_bias=delta_bias, delta_softplus=ctx.delta_softplus, h0=h0,
                              dlast=None if dlast is None else dlast.contiguous())
        return (g["dx"], g["dconv_w"], g["dconv_b"], g["ddelta"], g["dA"], g["dB"].to(B.dtype), g["dC"].to(C.dtype),
                g["dD"] if D is not None else None, g["dz"], g["ddelta_bias"] if delta_bias is not None else None,
                g["dh0"] if h0 is not None else None, None, None)


def selective_scan_conv(x: torch.Tensor, conv_w: torch.Tensor, conv_b: Optional[torch.Tensor], delta: torch.Tensor,
                        A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None,
                        delta_softplus: bool = False, h0: Optional[torch.Tensor] = None, state_chunk: int = 128):
    """Differentiable selective scan with the causal conv1d + SiLU in front
    (u = silu(conv1d(x))): returns (y, last_state)."""
    return _SelectiveScanConv.apply(x, conv_w, conv_b, delta, A, B, C, D, z, delta_bias, h0, delta_softplus,
                                    state_chunk)


class _OutProj(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, W):
        ctx.save_for_backward(y, W)
        return ssm_out_proj(y, W)

    @staticmethod
    def backward(ctx, dout):
        y, W = ctx.saved_tensors
        dy, dW = ssm_out_proj_bwd(y, W, dout.contiguous(), want_dy=ctx.needs_input_grad[0],
                                  want_dW=ctx.needs_input_grad[1])
        return dy, dW


def out_proj(y: torch.Tensor, W: torch.Tensor) -> torch.Tensor:
    """Differentiable output projection: out[b, t, m] = sum_k W[m, k] y[b, k, t]
    (y [b, d_inner, L] as the scan writes it, W [d_model, d_inner]); returns
    [b, L, d_model]."""
    return _OutProj.apply(y, W)


class _HeadScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, h0, g_head, lengths, scale):
        ctx.set_materialize_grads(False)
        o, last = ssm_head_scan_fwd(q, k, v, g=g, g_head=g_head, h0=h0, lengths=lengths, scale=scale)
        ctx.save_for_backward(q, k, v, g, h0, g_head, lengths)
        ctx.scale = scale
        return o, last

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dlast):
        q, k, v, g, h0, g_head, lengths = ctx.saved_tensors
        r = ssm_head_scan_bwd(q, k, v, v.new_zeros(v.shape) if do is None else _dense(do), g=g, g_head=g_head, h0=h0,
                              lengths=lengths, dlast=None if dlast is None else _dense(dlast), scale=ctx.scale,
                              want_dg=ctx.needs_input_grad[3], want_dh0=ctx.needs_input_grad[4])
        return r["dq"], r["dk"], r["dv"], r["dg"], r["dh0"], None, None, None


def head_scan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: Optional[torch.Tensor] = None,
              g_head: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
              lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None):
    """Differentiable head scan: returns (o, last_state).  g_head is a constant (a fixed decay per head takes no
    gradient); a learned one is expanded to g, where gradients are recorded at all."""
    if g_head is not None and g_head.requires_grad and torch.is_grad_enabled():
        raise ValueError("g_head takes no gradient: expand a learned decay to g [b, L, n_heads]")
    return _HeadScan.apply(q, k, v, g, h0, g_head, lengths, scale)


class _DeltaScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, g, h0, lengths, scale):
        ctx.set_materialize_grads(False)
        o, last = ssm_delta_scan_fwd(q, k, v, beta, g=g, h0=h0, lengths=lengths, scale=scale)
        ctx.save_for_backward(q, k, v, beta, g, h0, lengths)
        ctx.scale = scale
        return o, last

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dlast):
        q, k, v, beta, g, h0, lengths = ctx.saved_tensors
        r = ssm_delta_scan_bwd(q, k, v, v.new_zeros(v.shape) if do is None else _dense(do), beta, g=g, h0=h0,
                               lengths=lengths, dlast=None if dlast is None else _dense(dlast), scale=ctx.scale,
                               want_dbeta=ctx.needs_input_grad[3], want_dg=ctx.needs_input_grad[4],
                               want_dh0=ctx.needs_input_grad[5])
        return r["dq"], r["dk"], r["dv"], r["dbeta"], r["dg"], r["dh0"], None, None


def delta_scan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: Optional[torch.Tensor] = None,
               g: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
               lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None):
    """Differentiable delta scan: returns (o, last_state)."""
    return _DeltaScan.apply(q, k, v, beta, g, h0, lengths, scale)


class _GateNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, z, groups, eps, center, gate_first):
        ctx.save_for_backward(x, weight, z)
        ctx.opts = dict(groups=groups, eps=eps, center=center, gate_first=gate_first)
        return ssm_gate_norm(x, weight, z, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, z = ctx.saved_tensors
        dx, dw, dz = ssm_gate_norm_bwd(x, _dense(dy), weight, z, want_dweight=ctx.needs_input_grad[1], **ctx.opts)
        return dx, dw, dz, None, None, None, None


def gate_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, groups: int = 1,
              eps: float = 1e-5, center: bool = False, gate_first: bool = False) -> torch.Tensor:
    """Differentiable grouped norm of token rows [..., channels] with a SiLU gate."""
    return _GateNorm.apply(x, weight, z, groups, eps, center, gate_first)


class _AddNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, residual_dtype):
        ctx.set_materialize_grads(False)
        y, h = ssm_add_norm(x, residual, weight, eps=eps, residual_dtype=residual_dtype)
        ctx.save_for_backward(h, weight)
        ctx.eps, ctx.dtype = eps, x.dtype
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        # where y is not used dy is zero and so is what it gives
        dy = h.new_zeros(h.shape, dtype=ctx.dtype) if dy is None else _dense(dy)
        dx, dres, dw = ssm_add_norm_bwd(h, dy, weight, None if dh is None else _dense(dh), eps=ctx.eps, want_dx=need[0],
                                        want_dresidual=need[1], want_dweight=need[2])
        return dx, dres, dw, None, None


def add_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
             eps: float = 1e-5, residual_dtype: Optional[torch.dtype] = None):
    """Differentiable norm of token rows with the residual's addition: returns (y, h).  The gradients of x and of a
    residual of its dtype are one tensor."""
    return _AddNorm.apply(x, residual, weight, eps, residual_dtype)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, residual, act, keep):
        r = ssm_linear(x, W, bias, residual, act, return_pre=keep)
        out, pre = r if keep else (r, None)
        ctx.save_for_backward(x, W, pre)
        ctx.act = act
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x, W, pre = ctx.saved_tensors
        need = ctx.needs_input_grad
        dout = _dense(dout)
        dx = dW = db = None
        if any(need[:3]):
            dx, dW, db = ssm_linear_bwd(x, W, dout, pre, ctx.act, want_dx=need[0], want_dW=need[1], want_dbias=need[2])
        return dx, dW, db, dout if need[3] else None, None, None


def linear(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
           residual: Optional[torch.Tensor] = None, act: str = "none") -> torch.Tensor:
    """Differentiable linear layer on token rows [..., d_in] with its epilogue: act(x W^T + bias) + residual."""
    # the value before act is kept only where its slope will be asked for (needs_input_grad says so under no_grad too)
    keep = act != "none" and torch.is_grad_enabled() and any(
        isinstance(t, torch.Tensor) and t.requires_grad for t in (x, W, bias))
    return _Linear.apply(x, W, bias, residual, act, keep)
