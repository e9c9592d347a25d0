"""torch.autograd binding of the forward (ldn_chunk_fwd) and the backward
(ldn_backward): ``delta_rule(q, k, v, beta, gate, S0, mode=...)`` returns
(out, S_final) with gradients for q, k, v, beta, gate and S0; and of the operators
around it: ``add_rmsnorm``, ``short_conv`` and ``selective_scan``.  Argument
marshalling only: both directions run in the CUDA kernels of libldn.so.

Capturing a backward pass into a CUDA graph follows torch's rules for leaves: no
eager graph of the same leaves may be alive, since their gradient accumulators are
tied to the stream that made them.  The ``*_backward`` calls of ``mixer`` have no
such state and are captured freely.  The gradients of add_rmsnorm, short_conv and
selective_scan have no gradients of their own: asking for them raises.

The gradients of q, k and v are returned in their dtype (the kernel computes
them in fp32); beta, gate and S0 are fp32 throughout.  The output's gradient
reaches backward() in the output's dtype (autograd casts every incoming
gradient to the dtype of the tensor it belongs to), which is the inputs' dtype:
ldn_backward takes it in that dtype, and the conversion below only makes the
layout contiguous.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _native


def _mixer():
    # delta_rule needs no native torch layer: it is loaded where an operator of it is called
    from . import mixer
    return mixer


class _DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, gate, S0, mode):
        mode = _native.MODES.get(mode, mode)
        out, sf = _native.chunk_fwd(q, k, v, beta, gate, S0, mode=mode)
        ctx.mode = mode
        ctx.save_for_backward(q, k, v, beta, gate, S0)
        return out, sf

    @staticmethod
    def backward(ctx, dout, dsf):
        q, k, v, beta, gate, S0 = ctx.saved_tensors
        g = _native.backward(q, k, v, beta, gate, S0, dout.to(q.dtype).contiguous(),
                             None if dsf is None else dsf.float().contiguous(), mode=ctx.mode)
        return (g["dq"].to(q.dtype), g["dk"].to(k.dtype), g["dv"].to(v.dtype), g["dbeta"], g["dgate"],
                None if S0 is None else g["dS0"], None)


def delta_rule(q, k, v, beta, gate=None, S0=None, *, mode):
    """Chunkwise forward with autograd support (see ldn_chunk_fwd / ldn_backward
    in include/ldn.h).  Shapes as ``chunk_fwd``; returns (out, S_final)."""
    return _DeltaRule.apply(q, k, v, beta, gate, S0, mode)


class _AddRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, s = _mixer().add_rmsnorm(x, residual, weight, eps=eps)
        ctx.set_materialize_grads(False)
        ctx.eps = eps
        ctx.save_for_backward(s, weight)
        ctx.dtype, ctx.added = x.dtype, residual is not None
        return (y, s) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight = ctx.saved_tensors
        if dy is None:      # only the sum was used
            return (None if ds is None else ds.to(ctx.dtype)), ds, None, None
        g = _mixer().add_rmsnorm_backward(dy.contiguous(), s, weight, None if ds is None else ds.contiguous(),
                                          eps=ctx.eps)
        return g["dx"], g["dresidual"] if ctx.added else None, g["dweight"], None


def add_rmsnorm(x, residual, weight, *, eps=1e-6):
    """``mixer.add_rmsnorm`` with gradients for x, residual and weight; returns (y, s).  The
    gradient that reaches s joins y's in one kernel."""
    if residual is None:
        return _AddRmsNorm.apply(x, None, weight, eps), x
    return _AddRmsNorm.apply(x, residual, weight, eps)


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, lens, activation):
        ctx.set_materialize_grads(False)
        ctx.activation = activation
        ctx.save_for_backward(x, weight, bias, state, lens)
        return _mixer().short_conv(x, weight, bias, state, lens=lens, activation=activation)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dlast):
        x, weight, bias, state, lens = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        g = _mixer().short_conv_backward(x, weight, bias, dy, state, None if dlast is None else dlast.contiguous(),
                                         lens=lens, activation=ctx.activation)
        return g["dx"], g["dweight"], g["dbias"], g["dstate"], None, None


def short_conv(x, weight, bias=None, state=None, *, lens=None, activation=True):
    """``mixer.short_conv`` with gradients for x, weight, bias and state; returns (y, state_out)."""
    return _ShortConv.apply(x, weight, bias, state, lens, activation)


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, h0, lens, delta_softplus):
        ctx.set_materialize_grads(False)
        ctx.delta_softplus = delta_softplus
        y, h, states = _mixer().selective_scan(u, delta, A, B, C, D, z, delta_bias, h0, lens=lens,
                                               delta_softplus=delta_softplus, save_states=True)
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias, lens, states)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        u, delta, A, B, C, D, z, delta_bias, lens, states = ctx.saved_tensors
        dy = torch.zeros(u.shape, dtype=u.dtype, device=u.device) if dy is None else dy.contiguous()
        g = _mixer().selective_scan_backward(u, delta, A, B, C, D, z, delta_bias, states, dy,
                                             None if dh is None else dh.contiguous(), lens=lens,
                                             delta_softplus=ctx.delta_softplus)
        return (g["du"], g["ddelta"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddelta_bias"],
                g["dh0"] if ctx.needs_input_grad[8] else None, None, None)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, h0=None, *, lens=None, delta_softplus=True):
    """``mixer.selective_scan`` with gradients for every tensor but lens; returns (y, h_final).
    The forward keeps the state entering every 32 tokens for the gradient."""
    return _SelectiveScan.apply(u, delta, A, B, C, D, z, delta_bias, h0, lens, delta_softplus)
