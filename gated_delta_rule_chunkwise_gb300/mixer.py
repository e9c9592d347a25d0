"""The operators around a recurrent token mixer on torch CUDA tensors: ``add_rmsnorm``,
``add_rmsnorm_e4m3``, ``short_conv``, ``short_conv_step``, ``selective_scan``,
``selective_scan_step`` and the gradients ``add_rmsnorm_backward``,
``short_conv_backward``, ``selective_scan_backward`` (the C entry points ldn_add_rmsnorm*,
ldn_short_conv* and ldn_ssm_* of include/ldn.h).

Argument marshalling only: shape, type and device checks, strides, allocation of outputs
and workspaces.  Every call runs on the device of its tensors, on that device's current
stream, or on ``stream`` (a torch.cuda.Stream) when one is given: outputs and workspaces
are then allocated for that stream, and ordering it against the streams that made the
inputs and read the outputs is the caller's.
"""
from __future__ import annotations

import torch

from . import _native as _n

_F32, _BF16, _I32, _E4M3 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn
_CODES = {_F32: _n.LDN_F32, _BF16: _n.LDN_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice
_empty, _empty_like = torch.empty, torch.empty_like
_library = None


def _lib():
    global _library
    if _library is None:
        _library = _n.load()
    return _library


def _elsewhere(f, x, stream, args, kw):
    """f on the device of its first tensor x, and on `stream` where one is given."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{f.__name__}: the first argument must be a CUDA tensor")
    if stream is None:
        with torch.cuda.device(x.device):
            return f(*args, **kw)
    if stream.device != x.device:
        raise ValueError(f"{f.__name__}: stream is of {stream.device}, the tensors are on {x.device}")
    with torch.cuda.stream(stream):
        return f(*args, **kw)


def _away(x):
    """Whether x is not a tensor of the current device."""
    return not isinstance(x, torch.Tensor) or (d := x.get_device()) < 0 or d != _current()


def _code(t, name):
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return c


def _bad(t, name, shape, dtype, dev, rows=False):
    """Says what is wrong with an argument."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if rows:
        raise ValueError(f"{name} has strides {t.stride()}: rows must be contiguous and a constant distance apart")
    raise ValueError(f"{name} must be contiguous")


def _ptr(t, name, shape, dtype, dev):
    """The address of a contiguous tensor of this shape and type; None for None."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    _bad(t, name, shape, dtype, dev)


def _strided(t, name, shape, dtype, dev, lead):
    """(address, elements between rows): the `lead` leading dimensions count rows a constant
    distance apart, the others are one contiguous row."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _bad(t, name, shape, dtype, dev)
    s = t.stride()
    width = shape[-1]
    ok = s[-1] == 1 or width == 1
    if len(shape) > lead + 1:
        ok = ok and (s[lead] == width or shape[lead] == 1)
        width *= shape[lead]
    if lead == 1:
        ld = s[0] if shape[0] != 1 else width
    elif shape[1] == 1:
        ld = s[0] if shape[0] != 1 else width
    else:
        ld = s[1]
        ok = ok and (shape[0] == 1 or s[0] == shape[1] * ld)
    if not ok or ld < width:
        if t.numel():
            _bad(t, name, shape, dtype, dev, rows=True)
        ld = width      # no rows: no distance between them
    return t.data_ptr(), ld


def _done(status, what):
    if status != _n.LDN_OK:
        raise _n.LdnError(status, what)


def _workspace(nbytes, dev):
    return _empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


# ---- RMS norm with the residual's addition ----
def _norm_args(x, residual, weight, residual_out):
    """(addresses of x, residual, weight and the sum, the sum, type codes, device, rows, D)"""
    shape, dt = x.shape, x.dtype
    if not shape:
        raise ValueError("x must have at least one dimension")
    dev, D = x.get_device(), shape[-1]
    code = _code(x, "x")
    px, pw = _ptr(x, "x", shape, dt, dev), _ptr(weight, "weight", (D,), _F32, dev)
    if pw is None:
        raise TypeError("weight must be a CUDA tensor")
    rows = x.numel() // D if D else 0
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without residual")
        return px, None, pw, None, x, code, code, dev, rows, D
    rt = dt if residual.dtype is dt else residual.dtype
    rcode = code if rt is dt else _code(residual, "residual")
    pr = _ptr(residual, "residual", shape, rt, dev)
    if residual_out is None:
        residual_out = _empty_like(residual)
        po = residual_out.data_ptr()
    else:
        po = _ptr(residual_out, "residual_out", shape, rt, dev)
    return px, pr, pw, po, residual_out, code, rcode, dev, rows, D


def add_rmsnorm(x, residual, weight, *, eps=1e-6, out=None, residual_out=None, stream=None):
    """y = rmsnorm(s) * weight with s = x + residual (ldn_add_rmsnorm).

    x [..., D] float32 or bfloat16; residual of x's shape, in x's type or float32, or None
    (s = x); weight [D] float32.  Returns (y, s); s is `residual_out` (which may be
    `residual`: in place), a new tensor of residual's type, or x where there is none."""
    if stream is not None or _away(x):
        return _elsewhere(add_rmsnorm, x, stream, (x, residual, weight),
                          dict(eps=eps, out=out, residual_out=residual_out))
    px, pr, pw, po, s, code, rcode, dev, rows, D = _norm_args(x, residual, weight, residual_out)
    if out is None:
        out = _empty_like(x)
        py = out.data_ptr()
    else:
        py = _ptr(out, "out", x.shape, x.dtype, dev)
    st = _lib().ldn_add_rmsnorm(px, pr, pw, py, po, rows, D, code, rcode, eps, _raw_stream(dev))
    if st:
        raise _n.LdnError(st, "ldn_add_rmsnorm")
    return out, s


def add_rmsnorm_e4m3(x, residual, weight, *, eps=1e-6, group=0, out=None, scale=None, residual_out=None,
                     stream=None):
    """add_rmsnorm with the result in 8 bits (ldn_add_rmsnorm_e4m3): returns (q, scale, s),
    q float8_e4m3fn of x's shape, rmsnorm(s) * weight ~ q * scale.  group=0: one scale per
    row, scale [...]; group=128: one per 128 channels, scale [..., ceil(D / 128)]."""
    if stream is not None or _away(x):
        return _elsewhere(add_rmsnorm_e4m3, x, stream, (x, residual, weight),
                          dict(eps=eps, group=group, out=out, scale=scale, residual_out=residual_out))
    px, pr, pw, po, s, code, rcode, dev, rows, D = _norm_args(x, residual, weight, residual_out)
    shape = x.shape
    sshape = shape[:-1] if group == 0 else (*shape[:-1], (D + 127) // 128)
    if out is None:
        out = _empty_like(x, dtype=_E4M3)
        pq = out.data_ptr()
    else:
        pq = _ptr(out, "out", shape, _E4M3, dev)
    if scale is None:
        scale = _empty(sshape, dtype=_F32, device=x.device)
        ps = scale.data_ptr()
    else:
        ps = _ptr(scale, "scale", sshape, _F32, dev)
    st = _lib().ldn_add_rmsnorm_e4m3(px, pr, pw, pq, ps, po, rows, D, group, code, rcode, eps, _raw_stream(dev))
    if st:
        raise _n.LdnError(st, "ldn_add_rmsnorm_e4m3")
    return out, scale, s


def add_rmsnorm_backward(dy, s, weight, dsum=None, *, eps=1e-6, stream=None):
    """Gradients of add_rmsnorm (ldn_add_rmsnorm_backward).  dy: y's gradient, in y's type;
    s: what add_rmsnorm returned; dsum: the gradient that reaches s from elsewhere, or None.
    Returns a dict: dx in dy's type, dresidual in s's (the same tensor where the types are),
    dweight [D] float32."""
    if stream is not None or _away(dy):
        return _elsewhere(add_rmsnorm_backward, dy, stream, (dy, s, weight, dsum),
                          dict(eps=eps))
    dev, shape = dy.get_device(), dy.shape
    if dy.dim() < 1:
        raise ValueError("dy must have at least one dimension")
    D = shape[-1]
    code, rcode = _code(dy, "dy"), _code(s, "s")
    pdy, ps = _ptr(dy, "dy", shape, dy.dtype, dev), _ptr(s, "s", shape, s.dtype, dev)
    pw, pd = _ptr(weight, "weight", (D,), _F32, dev), _ptr(dsum, "dsum", shape, s.dtype, dev)
    rows = dy.numel() // max(D, 1)
    lib = _lib()
    dx = _empty_like(dy)
    dres = dx if code == rcode else _empty_like(s)
    dw = _empty((D,), dtype=_F32, device=dy.device)
    need = lib.ldn_add_rmsnorm_backward_workspace_size(rows, D)
    ws = _workspace(need, dy.device)
    _done(lib.ldn_add_rmsnorm_backward(pdy, ps, pw, pd, dx.data_ptr(), None if dres is dx else dres.data_ptr(),
                                       dw.data_ptr(), rows, D, code, rcode, eps, ws.data_ptr() if need else None,
                                       need, _raw_stream(dev)), "ldn_add_rmsnorm_backward")
    return dict(dx=dx, dresidual=dres, dweight=dw)


# ---- Short causal convolution ----
def _conv_args(x, weight, bias, lead):
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    if len(shape) != lead + 1:
        raise ValueError(f"x must have {lead + 1} dimensions, got {len(shape)}")
    code = _code(x, "x")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise TypeError("weight must be a CUDA tensor [C, width]")
    C, W = shape[-1], weight.shape[1]
    px, ldx = _strided(x, "x", shape, dt, dev, lead)
    return dev, C, W, code, px, ldx, _ptr(weight, "weight", (C, W), _F32, dev), _ptr(bias, "bias", (C,), _F32, dev)


def short_conv(x, weight, bias=None, state=None, *, lens=None, activation=True, out=None, state_out=None,
               stream=None):
    """Depthwise causal convolution and SiLU with a carried state (ldn_short_conv).

    x [B, T, C] float32 or bfloat16 (rows may be a slice of wider ones); weight [C, width]
    float32, last tap on the current token; bias [C] float32 or None; state
    [B, width-1, C] of x's type (the rows before, oldest first) or None for zeros; lens [B]
    int32 or None.  Returns (y, state_out); state_out may be `state`."""
    if stream is not None or _away(x):
        return _elsewhere(short_conv, x, stream, (x, weight, bias, state),
                          dict(lens=lens, activation=activation, out=out, state_out=state_out))
    dev, C, W, code, px, ldx, pw, pb = _conv_args(x, weight, bias, 2)
    B, T = x.shape[:2]
    sshape = (B, W - 1, C)
    pst = _ptr(state, "state", sshape, x.dtype, dev)
    pl = _ptr(lens, "lens", (B,), _I32, dev)
    if out is None:
        out = _empty((B, T, C), dtype=x.dtype, device=x.device)
        py = out.data_ptr()
    else:
        py = _ptr(out, "out", (B, T, C), x.dtype, dev)
    if state_out is None:
        state_out = _empty(sshape, dtype=x.dtype, device=x.device)
        pso = state_out.data_ptr()
    else:
        pso = _ptr(state_out, "state_out", sshape, x.dtype, dev)
    st = _lib().ldn_short_conv(px, ldx, pw, pb, pst, pl, py, pso, B, T, C, W, 1 if activation else 0, code,
                               _raw_stream(dev))
    if st:
        raise _n.LdnError(st, "ldn_short_conv")
    return out, state_out


def short_conv_step(x, weight, bias, state, *, activation=True, out=None, state_out=None, stream=None):
    """One token of short_conv for every sequence (ldn_short_conv_step): x [B, C], state
    [B, width-1, C], updated in place or, where given, written to `state_out`.  Returns y."""
    if stream is not None or _away(x):
        return _elsewhere(short_conv_step, x, stream, (x, weight, bias, state),
                          dict(activation=activation, out=out, state_out=state_out))
    dev, C, W, code, px, ldx, pw, pb = _conv_args(x, weight, bias, 1)
    B = x.shape[0]
    sshape = (B, W - 1, C)
    pst = _ptr(state, "state", sshape, x.dtype, dev)
    pso = pst if state_out is None else _ptr(state_out, "state_out", sshape, x.dtype, dev)
    if out is None:
        out = _empty((B, C), dtype=x.dtype, device=x.device)
        py = out.data_ptr()
    else:
        py = _ptr(out, "out", (B, C), x.dtype, dev)
    st = _lib().ldn_short_conv_step(px, ldx, pw, pb, pst, py, pso, B, C, W, 1 if activation else 0, code,
                                    _raw_stream(dev))
    if st:
        raise _n.LdnError(st, "ldn_short_conv_step")
    return out


def short_conv_backward(x, weight, bias, dy, state=None, dstate_out=None, *, lens=None, activation=True,
                        stream=None):
    """Gradients of short_conv (ldn_short_conv_backward) for y's gradient dy and, where
    given, the returned state's.  Returns a dict: dx, dstate in x's type (dstate None
    without a state), dweight, dbias float32 (dbias None without a bias)."""
    if stream is not None or _away(x):
        return _elsewhere(short_conv_backward, x, stream, (x, weight, bias, dy, state, dstate_out),
                          dict(lens=lens, activation=activation))
    dev, C, W, code, px, ldx, pw, pb = _conv_args(x, weight, bias, 2)
    B, T = x.shape[:2]
    sshape = (B, W - 1, C)
    pst, pds = _ptr(state, "state", sshape, x.dtype, dev), _ptr(dstate_out, "dstate_out", sshape, x.dtype, dev)
    pdy, pl = _ptr(dy, "dy", (B, T, C), x.dtype, dev), _ptr(lens, "lens", (B,), _I32, dev)
    lib, d = _lib(), x.device
    dx = _empty((B, T, C), dtype=x.dtype, device=d)
    dw = _empty((C, W), dtype=_F32, device=d)
    db = None if bias is None else _empty((C,), dtype=_F32, device=d)
    dst = None if state is None else _empty(sshape, dtype=x.dtype, device=d)
    need = lib.ldn_short_conv_backward_workspace_size(B, T, C, W)
    ws = _workspace(max(need, 16), d)
    _done(lib.ldn_short_conv_backward(px, ldx, pw, pb, pst, pl, pdy, pds, dx.data_ptr(), dw.data_ptr(),
                                      None if db is None else db.data_ptr(), None if dst is None else dst.data_ptr(),
                                      B, T, C, W, int(bool(activation)), code, ws.data_ptr(), need,
                                      _raw_stream(dev)), "ldn_short_conv_backward")
    return dict(dx=dx, dweight=dw, dbias=db, dstate=dst)


# ---- Selective state space scan ----
def _ssm_args(u, delta, A, B, C, D, z, delta_bias, lead):
    shape, dt, dev = u.shape, u.dtype, u.get_device()
    if len(shape) != lead + 1:
        raise ValueError(f"u must have {lead + 1} dimensions, got {len(shape)}")
    code, Dm = _code(u, "u"), shape[-1]
    if not isinstance(B, torch.Tensor) or B.dim() != lead + 2:
        raise ValueError(f"B must be a CUDA tensor of {lead + 2} dimensions")
    bshape = B.shape
    G, N = bshape[-2:]
    if bshape[:lead] != shape[:lead]:
        _bad(B, "B", (*shape[:lead], G, N), dt, dev)
    pu, ldu = _strided(u, "u", shape, dt, dev, lead)
    pd, ldd = _strided(delta, "delta", shape, dt, dev, lead)
    pB, ldB = _strided(B, "B", bshape, dt, dev, lead)
    pC, ldC = _strided(C, "C", bshape, dt, dev, lead)
    pz, ldz = (None, Dm) if z is None else _strided(z, "z", shape, dt, dev, lead)
    pA = _ptr(A, "A", (Dm, N), _F32, dev)
    pD, pb = _ptr(D, "D", (Dm,), _F32, dev), _ptr(delta_bias, "delta_bias", (Dm,), _F32, dev)
    return (pu, ldu, pd, ldd, pA, pB, ldB, pC, ldC, pD, pz, ldz, pb), dev, Dm, N, G, code


def chunk_states_shape(B, T, D, N):
    """The shape of the states a scan of these sizes saves for its gradient."""
    return B, (T + 31) // 32, D, N


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, h0=None, *, delta_softplus=True, lens=None,
                   save_states=False, out=None, h_final=None, workspace=None, stream=None):
    """Selective state space scan over whole sequences (ldn_ssm_scan).

    u, delta, z [B, T, Dm] and B, C [B, T, G, N] float32 or bfloat16, one type (rows may be
    slices of wider ones); A [Dm, N], D, delta_bias [Dm], h0 [B, Dm, N] float32; lens [B]
    int32; D, z, delta_bias, h0, lens may be None.  Returns (y, h_final), with
    save_states=True (y, h_final, states) for selective_scan_backward.  `workspace`: a uint8
    tensor for the segments of a scan over few channels; None allocates what
    ldn_ssm_scan_workspace_size asks for, an empty one runs unsplit."""
    if stream is not None or _away(u):
        return _elsewhere(selective_scan, u, stream, (u, delta, A, B, C, D, z, delta_bias, h0),
                          dict(delta_softplus=delta_softplus, lens=lens, save_states=save_states, out=out, h_final=h_final, workspace=workspace))
    args, dev, Dm, N, G, code = _ssm_args(u, delta, A, B, C, D, z, delta_bias, 2)
    nb, T = u.shape[:2]
    hshape = (nb, Dm, N)
    ph, pl = _ptr(h0, "h0", hshape, _F32, dev), _ptr(lens, "lens", (nb,), _I32, dev)
    d, lib = u.device, _lib()
    if out is None:
        out = _empty((nb, T, Dm), dtype=u.dtype, device=d)
    if h_final is None:
        h_final = _empty(hshape, dtype=_F32, device=d)
    py, pf = _ptr(out, "out", (nb, T, Dm), u.dtype, dev), _ptr(h_final, "h_final", hshape, _F32, dev)
    states = _empty(chunk_states_shape(nb, T, Dm, N), dtype=_F32, device=d) if save_states else None
    if workspace is None:
        workspace = _workspace(lib.ldn_ssm_scan_workspace_size(nb, T, Dm, N, G), d)
    else:
        _ptr(workspace, "workspace", workspace.shape, torch.uint8, dev)
    nws = 0 if workspace is None else workspace.numel()
    _done(lib.ldn_ssm_scan(*args, ph, pl, py, pf, states.data_ptr() if save_states else None, nb, T, Dm, N, G,
                           int(bool(delta_softplus)), code, workspace.data_ptr() if nws else None, nws,
                           _raw_stream(dev)), "ldn_ssm_scan")
    return (out, h_final, states) if save_states else (out, h_final)


def selective_scan_step(u, delta, A, B, C, D, z, delta_bias, h, *, delta_softplus=True, out=None, h_out=None,
                        stream=None):
    """One token of selective_scan for every sequence (ldn_ssm_step): u, delta, z [B, Dm],
    B, C [B, G, N], h [B, Dm, N] float32, updated in place or, where given, written to
    `h_out`.  Returns y."""
    if stream is not None or _away(u):
        return _elsewhere(selective_scan_step, u, stream, (u, delta, A, B, C, D, z, delta_bias, h),
                          dict(delta_softplus=delta_softplus, out=out, h_out=h_out))
    args, dev, Dm, N, G, code = _ssm_args(u, delta, A, B, C, D, z, delta_bias, 1)
    nb = u.shape[0]
    hshape = (nb, Dm, N)
    ph = _ptr(h, "h", hshape, _F32, dev)
    po = ph if h_out is None else _ptr(h_out, "h_out", hshape, _F32, dev)
    if out is None:
        out = _empty((nb, Dm), dtype=u.dtype, device=u.device)
        py = out.data_ptr()
    else:
        py = _ptr(out, "out", (nb, Dm), u.dtype, dev)
    st = _lib().ldn_ssm_step(*args, ph, po, py, nb, Dm, N, G, 1 if delta_softplus else 0, code, _raw_stream(dev))
    if st:
        raise _n.LdnError(st, "ldn_ssm_step")
    return out


def selective_scan_backward(u, delta, A, B, C, D, z, delta_bias, states, dy, dh_final=None, *, delta_softplus=True,
                            lens=None, stream=None):
    """Gradients of selective_scan (ldn_ssm_backward) from the states it saved, for y's
    gradient dy [B, T, Dm] and, where given, the final state's.  Returns a dict: du, ddelta,
    dz, dB, dC in u's type; dA, dD, ddelta_bias, dh0 float32; None in the place of a
    gradient whose input is None."""
    if stream is not None or _away(u):
        return _elsewhere(selective_scan_backward, u, stream, (u, delta, A, B, C, D, z, delta_bias, states, dy, dh_final),
                          dict(delta_softplus=delta_softplus, lens=lens))
    args, dev, Dm, N, G, code = _ssm_args(u, delta, A, B, C, D, z, delta_bias, 2)
    nb, T = u.shape[:2]
    hshape = (nb, Dm, N)
    ps = _ptr(states, "states", chunk_states_shape(nb, T, Dm, N), _F32, dev)
    pl = _ptr(lens, "lens", (nb,), _I32, dev)
    pdy, pdh = _ptr(dy, "dy", u.shape, u.dtype, dev), _ptr(dh_final, "dh_final", hshape, _F32, dev)
    d, lib, e = u.device, _lib(), u.dtype
    new = lambda shape, dtype: _empty(shape, dtype=dtype, device=d)  # noqa: E731
    g = dict(du=new(u.shape, e), ddelta=new(u.shape, e), dA=new((Dm, N), _F32), dB=new(B.shape, e), dC=new(B.shape, e),
             dD=None if D is None else new((Dm,), _F32), dz=None if z is None else new(u.shape, e),
             ddelta_bias=None if delta_bias is None else new((Dm,), _F32), dh0=new(hshape, _F32))
    need = lib.ldn_ssm_backward_workspace_size(nb, T, Dm, N, G)
    ws = _workspace(max(need, 16), d)
    _done(lib.ldn_ssm_backward(*args, ps, pl, pdy, pdh, *(None if t is None else t.data_ptr() for t in g.values()),
                               nb, T, Dm, N, G, int(bool(delta_softplus)), code, ws.data_ptr(), need,
                               _raw_stream(dev)), "ldn_ssm_backward")
    return g
