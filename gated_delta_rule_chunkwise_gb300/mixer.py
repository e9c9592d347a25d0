"""The operators around a recurrent token mixer on torch CUDA tensors: ``add_rmsnorm``,
``add_rmsnorm_e4m3``, ``short_conv``, ``short_conv_step``, ``selective_scan``,
``selective_scan_step``, ``gated_add_rmsnorm``, ``linear``, ``linear_e4m3`` and the gradients
``add_rmsnorm_backward``, ``short_conv_backward``, ``selective_scan_backward``,
``gated_add_rmsnorm_backward``, ``linear_backward`` (the C entry points ldn_add_rmsnorm*,
ldn_short_conv*, ldn_ssm_*, ldn_gated_add_rmsnorm* and ldn_linear* of include/ldn.h).

Argument marshalling only, in native code (csrc/torch/, lib/_ldn_torch.so): shape, type and
device checks, strides, allocation of outputs and workspaces.  Wrong types raise TypeError,
wrong shapes, strides or devices ValueError, and what the C entry point refuses
``LdnError``.  Every call runs on the device of its tensors, on that device's current
stream, or on ``stream`` (a torch.cuda.Stream) when one is given: outputs and workspaces are
then allocated for that stream, the arguments' memory is kept from reuse until it is done
with them, and ordering it against the streams that made the inputs and read the outputs is
the caller's.

None of these calls records gradients: ``autograd`` has add_rmsnorm, short_conv,
selective_scan, gated_add_rmsnorm and linear with them.  The calls of the same names here, and
add_rmsnorm_e4m3 and linear_e4m3, warn (UserWarning) where gradients are being recorded and an argument requires one; the others,
for single tokens and gradients, do not.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from . import _native as _n

LIB_PATH = os.path.join(os.path.dirname(_n.LIB_PATH), "_ldn_torch.so")


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"_ldn_torch.so not found at {LIB_PATH}; run __graft_entry__.build() "
                           "(or gated_delta_rule_chunkwise_gb300.build.build()) first")
    _n.load()
    loader = importlib.machinery.ExtensionFileLoader("_ldn_torch", LIB_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_ldn_torch", loader))
    loader.exec_module(module)
    module.set_error(_n.LdnError)
    return module


_core = _load()
_norm, _norm_bwd = _core.add_rmsnorm, _core.add_rmsnorm_backward
_conv, _conv_step, _conv_bwd = _core.short_conv, _core.short_conv_step, _core.short_conv_backward
_gated, _gated_bwd = _core.gated_add_rmsnorm, _core.gated_add_rmsnorm_backward
_linear, _linear_e4m3, _linear_bwd = _core.linear, _core.linear_e4m3, _core.linear_backward
_ACTIVATIONS = {None: _n.LDN_ACT_NONE, "silu": _n.LDN_ACT_SILU, "gelu": _n.LDN_ACT_GELU}
_scan, _scan_step, _scan_bwd = _core.selective_scan, _core.selective_scan_step, _core.selective_scan_backward


def _call(f, stream, x, *args):
    """f(x, ...) on `stream`, or on x's device where that is not the current one."""
    if stream is None:
        r = f(x, *args)
        if r is not None:
            return r
        with torch.cuda.device(x.device):
            return f(x, *args)
    if not isinstance(stream, torch.cuda.Stream) or not isinstance(x, torch.Tensor) or stream.device != x.device:
        raise ValueError(f"{f.__name__}: stream must be a torch.cuda.Stream of the first tensor's device")
    with torch.cuda.stream(stream):
        r = f(x, *args)
    for t in (x, *args):    # freed after the call, their memory waits for this stream
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return r


# ---- RMS norm with the residual's addition ----
def add_rmsnorm(x, residual, weight, *, eps=1e-6, out=None, residual_out=None, stream=None):
    """y = rmsnorm(s) * weight with s = x + residual (ldn_add_rmsnorm).

    x [..., D] float32 or bfloat16; residual of x's shape, in x's type or float32, or None
    (s = x); weight [D] float32.  Returns (y, s); s is `residual_out` (which may be
    `residual`: in place), a new tensor of residual's type, or x where there is none."""
    return _call(_norm, stream, x, residual, weight, eps, out, residual_out)


def add_rmsnorm_e4m3(x, residual, weight, *, eps=1e-6, group=0, out=None, scale=None, residual_out=None, stream=None):
    """add_rmsnorm with the result in 8 bits (ldn_add_rmsnorm_e4m3): returns (q, scale, s),
    q float8_e4m3fn of x's shape, rmsnorm(s) * weight ~ q * scale.  group=0: one scale per
    row, scale [...]; group=128: one per 128 channels, scale [..., ceil(D / 128)]."""
    return _call(_norm, stream, x, residual, weight, eps, out, residual_out, group, scale)


def add_rmsnorm_backward(dy, s, weight, dsum=None, *, eps=1e-6, stream=None):
    """Gradients of add_rmsnorm (ldn_add_rmsnorm_backward).  dy: y's gradient, in y's type;
    s: what add_rmsnorm returned; dsum: the gradient that reaches s from elsewhere, or None.
    Returns a dict: dx in dy's type, dresidual in s's (the same tensor where the types are),
    dweight [D] float32."""
    return _call(_norm_bwd, stream, dy, s, weight, dsum, eps)


# ---- Short causal convolution ----
def short_conv(x, weight, bias=None, state=None, *, lens=None, activation=True, out=None, state_out=None,
               stream=None):
    """Depthwise causal convolution and SiLU with a carried state (ldn_short_conv).

    x [B, T, C] float32 or bfloat16 (rows may be a slice of wider ones); weight [C, width]
    float32, last tap on the current token; bias [C] float32 or None; state
    [B, width-1, C] of x's type (the rows before, oldest first) or None for zeros; lens [B]
    int32 or None.  Returns (y, state_out); state_out may be `state`."""
    return _call(_conv, stream, x, weight, bias, state, lens, activation, out, state_out)


def short_conv_step(x, weight, bias, state, *, activation=True, out=None, state_out=None, stream=None):
    """One token of short_conv for every sequence (ldn_short_conv_step): x [B, C], state
    [B, width-1, C], updated in place or, where given, written to `state_out`.  Returns y."""
    return _call(_conv_step, stream, x, weight, bias, state, activation, out, state_out)


def short_conv_backward(x, weight, bias, dy, state=None, dstate_out=None, *, lens=None, activation=True,
                        stream=None):
    """Gradients of short_conv (ldn_short_conv_backward) for y's gradient dy and, where
    given, the returned state's.  Returns a dict: dx, dstate in x's type (dstate None
    without a state), dweight, dbias float32 (dbias None without a bias)."""
    return _call(_conv_bwd, stream, x, weight, bias, dy, state, dstate_out, lens, activation)


# ---- Selective state space scan ----
def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, h0=None, *, delta_softplus=True, lens=None,
                   save_states=False, out=None, h_final=None, workspace=None, stream=None):
    """Selective state space scan over whole sequences (ldn_ssm_scan).

    u, delta, z [B, T, Dm] and B, C [B, T, G, N] float32 or bfloat16, one type (rows may be
    slices of wider ones); A [Dm, N], D, delta_bias [Dm], h0 [B, Dm, N] float32; lens [B]
    int32; D, z, delta_bias, h0, lens may be None.  Returns (y, h_final), with
    save_states=True (y, h_final, states) for selective_scan_backward.  `workspace`: a uint8
    tensor for the segments of a scan over few channels; None allocates what
    ldn_ssm_scan_workspace_size asks for, an empty one runs unsplit."""
    return _call(_scan, stream, u, delta, A, B, C, D, z, delta_bias, h0, delta_softplus, lens, save_states, out,
                 h_final, workspace)


def selective_scan_step(u, delta, A, B, C, D, z, delta_bias, h, *, delta_softplus=True, out=None, h_out=None,
                        stream=None):
    """One token of selective_scan for every sequence (ldn_ssm_step): u, delta, z [B, Dm],
    B, C [B, G, N], h [B, Dm, N] float32, updated in place or, where given, written to
    `h_out`.  Returns y."""
    return _call(_scan_step, stream, u, delta, A, B, C, D, z, delta_bias, h, delta_softplus, out, h_out)


def selective_scan_backward(u, delta, A, B, C, D, z, delta_bias, states, dy, dh_final=None, *, delta_softplus=True,
                            lens=None, stream=None):
    """Gradients of selective_scan (ldn_ssm_backward) from the states it saved, for y's
    gradient dy [B, T, Dm] and, where given, the final state's.  Returns a dict: du, ddelta,
    dz, dB, dC in u's type; dA, dD, ddelta_bias, dh0 float32; None in the place of a
    gradient whose input is None."""
    return _call(_scan_bwd, stream, u, delta, A, B, C, D, z, delta_bias, states, dy, dh_final, delta_softplus, lens)


# ---- Norms around a block with its gate and the residual's scale ----
def gated_add_rmsnorm(x, residual, weight=None, post_weight=None, gate=None, *, residual_scale=1.0,
                      gate_sigmoid=False, eps=1e-6, out=None, residual_out=None, stream=None):
    """From a block's output to the next block's input (ldn_gated_add_rmsnorm):
    s = residual_scale * residual + g * n with n = rmsnorm(x) * post_weight (x without one) and
    g = gate or, with gate_sigmoid, sigmoid(gate) (1 without one); y = rmsnorm(s) * weight.

    x [..., D] float32 or bfloat16; residual of x's shape, in x's type or float32; weight,
    post_weight [D] float32 or None; gate in x's type or float32: [D], or x's number of
    dimensions, as large as x's up to some dimension, 1 from there on and D last ([B, 1, D] for
    x [B, T, D] is one per sequence), or None.  Returns (y, s): y None without weight; s is
    `residual_out` (which may be `residual`: in place) or a new tensor of residual's type."""
    return _call(_gated, stream, x, residual, weight, post_weight, gate, residual_scale, gate_sigmoid, eps, out,
                 residual_out)


def gated_add_rmsnorm_backward(dy, x, s, weight=None, post_weight=None, gate=None, dsum=None, *, residual_scale=1.0,
                               gate_sigmoid=False, eps=1e-6, stream=None):
    """Gradients of gated_add_rmsnorm (ldn_gated_add_rmsnorm_backward).  dy: y's gradient in x's
    type, None exactly where weight is; s: what gated_add_rmsnorm returned; dsum: the gradient
    that reaches s from elsewhere, or None.  Returns a dict: dx in x's type, dresidual in s's,
    dgate in gate's type and shape, dweight, dpost_weight [D] float32; None in the place of a
    gradient whose input is None."""
    return _call(_gated_bwd, stream, x, dy, s, weight, post_weight, gate, dsum, residual_scale, gate_sigmoid, eps)


# ---- Projections ----
def _activation(name):
    try:
        return _ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be None, 'silu' or 'gelu', got {name!r}") from None


def linear(x, weight, bias=None, residual=None, *, activation=None, save_z=False, out=None, stream=None):
    """y = act(x weight^T + bias) + residual (ldn_linear); act None, 'silu' or 'gelu' (z Phi(z)).

    x [..., K] float32 or bfloat16 (rows may be a slice of wider ones); weight [N, K] of x's
    type (rows likewise); bias [N] of x's type or None; residual [..., N] in x's type or float32,
    or None.  y [..., N] is `out` (which may be `residual`: in place) or a new tensor, in
    residual's type, x's without one.  With save_z=True returns (y, z), z = x weight^T + bias in
    x's type for linear_backward."""
    return _call(_linear, stream, x, weight, bias, residual, _activation(activation), save_z, out)


def linear_e4m3(x, x_scale, weight, weight_scale, bias=None, residual=None, *, activation=None, out=None, stream=None):
    """linear from 8 bits (ldn_linear_e4m3): x [..., K] and weight [N, K] float8_e4m3fn with
    x_scale [...] and weight_scale [N] float32, one scale a row (add_rmsnorm_e4m3's with
    group=0); bias [N] bfloat16 or None; residual [..., N] bfloat16 or float32, or None.  y in
    residual's type, bfloat16 without one."""
    return _call(_linear_e4m3, stream, x, x_scale, weight, weight_scale, bias, residual, _activation(activation), out)


def linear_backward(dy, x, weight, z=None, *, activation=None, bias=False, dx=True, dweight=True, stream=None):
    """Gradients of linear (ldn_linear_backward) for y's gradient dy [..., N], in x's type or
    float32; the residual's gradient is dy itself.  z: what linear(save_z=True) returned, needed
    with an activation.  Returns a dict: dx, dweight, dbias in x's type; dbias None where `bias`
    is false, dx and dweight likewise."""
    return _call(_linear_bwd, stream, x, dy, weight, z, _activation(activation), dx, dweight, bias)
