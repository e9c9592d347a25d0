"""64-bit plain implementations of the operators that join blocks (the norms around a block with
its gate and the residual's scale, the projections), their gradients, and bounds of the error that
the kernels' arithmetic may have (numpy, CPU)."""
import math

import numpy as np

from tests._mixer_ref import HALF, U, e_sig, sigmoid

_erf = np.vectorize(math.erf, otypes=[float])


# ---- norms around a block ----
def root(v, eps):
    return 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def spread(gate, shape):
    """The gate's values for every element: gate [D], [B, 1, D], [B, T, D] or None."""
    return np.ones(shape) if gate is None else np.broadcast_to(gate, shape)


def gated(x, r, w, wp, gate, scale, sig, eps, s=None):
    """(s, y) before rounding; y of the given s where there is one."""
    n = x if wp is None else x * root(x, eps) * wp
    g = spread(gate, x.shape)
    own = scale * r + (sigmoid(g) if sig and gate is not None else g) * n
    s = own if s is None else s
    return own, None if w is None else s * root(s, eps) * w


def fold(v, shape):
    """Sums of v over what a gate of this shape is shared by."""
    if len(shape) == 1:
        return v.reshape(-1, v.shape[-1]).sum(0)
    for i, n in enumerate(shape):
        if n == 1 and v.shape[i] != 1:
            v = v.sum(i, keepdims=True)
    return v


def _norm_grad(dn, v, w, rho):
    wd = w * dn
    return rho * (wd - v * rho ** 2 * (wd * v).mean(-1, keepdims=True))


def gated_bwd(dy, x, s, w, wp, gate, dsum, scale, sig, eps):
    g = spread(gate, x.shape)
    gv = sigmoid(g) if sig and gate is not None else g
    out = {}
    ds = np.zeros(x.shape) if dsum is None else dsum
    lead = tuple(range(x.ndim - 1))
    if w is not None:
        rho = root(s, eps)
        out["dweight"] = (dy * s * rho).sum(lead)
        ds = ds + _norm_grad(dy, s, w, rho)
    out["dresidual"] = scale * ds
    n = x if wp is None else x * root(x, eps) * wp
    if gate is not None:
        out["dgate"] = fold(ds * n * (gv * (1 - gv) if sig else 1), gate.shape)
    dn = ds * gv
    if wp is not None:
        rho = root(x, eps)
        out["dpost_weight"] = (dn * x * rho).sum(lead)
        dn = _norm_grad(dn, x, wp, rho)
    out["dx"] = dn
    return out


def gated_bounds(x, r, w, wp, gate, scale, sig, eps, s, dtype, res, gtype=None, dy=None, dsum=None):
    """Absolute error bounds of s, y and, given dy or dsum, of the gradients; y and the gradients
    from s as it was stored.  k roundings of fp32 a sum over a row: a chain of D / 256 and a tree,
    halved by the root; a dozen for what is formed of it."""
    D = x.shape[-1]
    k = (24 + D / 256) * U
    own, y = gated(x, r, w, wp, gate, scale, sig, eps, s)
    g = spread(gate, x.shape)
    gv = sigmoid(g) if sig and gate is not None else g
    eg = e_sig(g) * gv if sig and gate is not None else 0.0
    n = x if wp is None else x * root(x, eps) * wp
    b = {"s": HALF[res] * np.abs(own) + k * (np.abs(scale * r) + np.abs(gv * n)) + eg * np.abs(n)}
    if w is not None:
        b["y"] = np.abs(y) * (HALF[dtype] + k) + 1e-30
    if dy is None and dsum is None:
        return b
    ds, eds = (np.zeros(x.shape),) * 2 if dsum is None else (dsum, np.zeros(x.shape))
    rows = x.size // D
    run = (64 + rows / 100) * U + k     # a column's chain over the rows of a block, and of the blocks
    lead = tuple(range(x.ndim - 1))
    mean = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    if w is not None:
        rho = root(s, eps)
        mag = rho * (np.abs(w * dy) + np.abs(s) * rho ** 2 * mean(np.abs(w * dy * s)))
        b["dweight"] = run * np.abs(dy * s * rho).sum(lead) + 1e-30
        ds = ds + _norm_grad(dy, s, w, rho)
        eds = k * (mag + np.abs(ds))
    b["dresidual"] = np.abs(scale) * eds + (HALF[res] + U) * np.abs(scale * ds) + 1e-30
    if gate is not None:
        slope = gv * (1 - gv) if sig else np.ones(x.shape)
        eslope = 2 * e_sig(g) * gv if sig else 0.0
        mag = np.abs(ds * n) * slope
        bound = fold(slope * (eds * np.abs(n)) + run * mag + np.abs(ds * n) * eslope, gate.shape)
        b["dgate"] = bound + HALF[gtype] * np.abs(fold(ds * n * slope, gate.shape)) + 1e-30
    dn = ds * gv
    edn = eds * np.abs(gv) + eg * np.abs(ds) + U * np.abs(dn)
    dx = dn
    if wp is not None:
        rho = root(x, eps)
        b["dpost_weight"] = (np.abs(x * rho) * edn + run * np.abs(dn * x * rho)).sum(lead) + 1e-30
        dx = _norm_grad(dn, x, wp, rho)
        through = lambda v: rho * (np.abs(wp) * v + np.abs(x) * rho ** 2 * mean(np.abs(wp * x) * v))  # noqa: E731
        edn = through(edn) + k * through(np.abs(dn))
    b["dx"] = edn + HALF[dtype] * np.abs(dx) + 1e-30
    return b


# ---- projections ----
def act(z, name):
    return z * sigmoid(z) if name == "silu" else z * 0.5 * (1 + _erf(z / math.sqrt(2))) if name == "gelu" else z


def dact(z, name):
    if name == "silu":
        s = sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return np.ones_like(z)


def linear(x, w, b, r, name):
    z = x @ w.T + (0 if b is None else b)
    return act(z, name) + (0 if r is None else r), z


def linear_bwd(dy, x, w, z, name):
    dz = dy * dact(z, name)
    return dict(dx=dz @ w, dweight=dz.T @ x, dbias=dz.sum(0)), dz


def summed(mag, k, kept):
    """Bound of a sum over k products of magnitude sum `mag` in tensor memory: 16 products a step,
    each step and the tree within it cut off at up to a step of fp32.  kept: an fp32 result, of chunks
    of at most 1024 that are added in registers, rounded to nearest, and of fp32 factors without the
    smallest three of their nine products (2^-25)."""
    steps = min(k, 1024) / 16 if kept else k / 16
    return mag * ((steps + 32) * 2 * U + (k / 256 * U + U if kept else 0))


SLOPE, BEND = 1.13, 0.8     # of silu and gelu: the largest first and second derivatives


def linear_bounds(x, w, b, r, name, dtype, out, dy=None):
    """Absolute error bounds of y and z and, given dy, of dx, dweight, dbias."""
    y, z = linear(x, w, b, r, name)
    K, N = x.shape[1], w.shape[0]
    ez = summed(np.abs(x) @ np.abs(w).T, K, out == "f32") + U * np.abs(z) + (0 if b is None else U * np.abs(b))
    # the activation's own arithmetic: e^-z and a quotient, or erf to two steps of 1 and its product
    ea = 0.0 if name is None else e_sig(z) * np.abs(z) + 4 * U * np.abs(z)
    ey = (SLOPE if name else 1.0) * ez + ea + (0 if r is None else U * np.abs(y)) + HALF[out] * np.abs(y)
    bounds = dict(y=ey + 1e-30, z=ez + HALF[dtype] * np.abs(z) + 1e-30)
    if dy is None:
        return bounds
    g, dz = linear_bwd(dy, x, w, z, name)
    # from z as it was stored; dz is rounded for its two products
    edz = 0.0 if name is None else np.abs(dy) * (BEND * bounds["z"] + e_sig(z) * (1 + np.abs(z)) + 8 * U)
    edz = edz + U * np.abs(dz)
    eround = edz + (HALF[dtype] * np.abs(dz) if dtype == "bf16" else 0.0)
    kept = dtype == "f32"
    bounds["dx"] = eround @ np.abs(w) + summed(np.abs(dz) @ np.abs(w), N, kept) + HALF[dtype] * np.abs(g["dx"]) + 1e-30
    bounds["dweight"] = (eround.T @ np.abs(x) + summed(np.abs(dz).T @ np.abs(x), x.shape[0], kept)
                         + HALF[dtype] * np.abs(g["dweight"]) + 1e-30)
    run = (64 + x.shape[0] / 8) * U
    bounds["dbias"] = edz.sum(0) + run * np.abs(dz).sum(0) + HALF[dtype] * np.abs(g["dbias"]) + 1e-30
    return bounds
