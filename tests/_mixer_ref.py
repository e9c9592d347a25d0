"""64-bit plain implementations of the operators around a token mixer, token by token from
their definitions (numpy, CPU), and the inputs of their tests."""
import numpy as np


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def silu(x):
    return x * sigmoid(x)


def dsilu(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


# ---- RMS norm with the residual's addition ----
def norm(s, w, eps):
    s = s.astype(np.float64)
    return s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * w


def norm_bwd(dy, s, w, dsum, eps):
    s, dy = s.astype(np.float64), dy.astype(np.float64)
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    wd = w * dy
    ds = r * (wd - s * r * r * (wd * s).mean(-1, keepdims=True))
    return ds + (0 if dsum is None else dsum), (dy * s * r).sum(0)


def e4m3(v):
    """v rounded to e4m3 (to nearest even, saturating), as float64."""
    v = np.clip(v, -448.0, 448.0)
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    return np.clip(np.round(v / step) * step, -448.0, 448.0)


def groups_of(y, group):
    """max |y| of each group and the scales: [rows][n]."""
    D = y.shape[-1]
    g = group or D
    n = -(-D // g)
    p = np.zeros((*y.shape[:-1], n * g))
    p[..., :D] = np.abs(y)
    return np.maximum(p.reshape(*y.shape[:-1], n, g).max(-1), 2.0 ** -100) / 448.0


# ---- short convolution ----
def conv(x, w, b, state, lens, act):
    """y, pre-activation and the last rows; x [B,T,C], lens a list."""
    B, T, C = x.shape
    W = w.shape[1]
    y, p = np.zeros((B, T, C)), np.zeros((B, T, C))
    last = np.zeros((B, W - 1, C))
    for i in range(B):
        head = np.zeros((W - 1, C)) if state is None else state[i]
        seq = np.concatenate([head, x[i, :lens[i]]]).astype(np.float64)
        for t in range(lens[i]):
            p[i, t] = (seq[t:t + W].T * w).sum(1) + (0 if b is None else b)
        y[i, :lens[i]] = silu(p[i, :lens[i]]) if act else p[i, :lens[i]]
        last[i] = seq[lens[i]:lens[i] + W - 1]
    return y, p, last


def conv_bwd(x, w, b, state, lens, act, dy, dlast):
    B, T, C = x.shape
    W = w.shape[1]
    _, p, _ = conv(x, w, b, state, lens, act)
    dx, dst = np.zeros((B, T, C)), np.zeros((B, W - 1, C))
    dw, db = np.zeros((C, W)), np.zeros(C)
    for i in range(B):
        n = lens[i]
        head = np.zeros((W - 1, C)) if state is None else state[i]
        seq = np.concatenate([head, x[i, :n]]).astype(np.float64)
        dseq = np.zeros_like(seq)
        for t in range(n):
            dp = dy[i, t].astype(np.float64) * (dsilu(p[i, t]) if act else 1.0)
            dw += dp[:, None] * seq[t:t + W].T
            db += dp
            dseq[t:t + W] += (dp[:, None] * w).T
        if dlast is not None:
            dseq[n:n + W - 1] += dlast[i]
        dst[i], dx[i, :n] = dseq[:W - 1], dseq[W - 1:]
    return dx, dw, db, dst


# ---- selective scan ----
def _wide(m, D):
    """[G, N] to [D, N]"""
    return np.repeat(m.astype(np.float64), D // m.shape[0], axis=0)


def scan(p, lens):
    """y and every state [B][T+1][D][N] for a dict of numpy inputs."""
    u, A = p["u"].astype(np.float64), p["A"].astype(np.float64)
    B, T, D = u.shape
    N = A.shape[1]
    raw = p["delta"].astype(np.float64) + (0 if p["bias"] is None else p["bias"])
    dt = softplus(raw) if p["softplus"] else raw
    h = np.zeros((B, T + 1, D, N))
    if p["h0"] is not None:
        h[:, 0] = p["h0"]
    pre = np.zeros((B, T, D))
    for i in range(B):
        for t in range(T):
            if t >= lens[i]:
                h[i, t + 1] = h[i, t]
                continue
            h[i, t + 1] = (np.exp(dt[i, t][:, None] * A) * h[i, t]
                           + (dt[i, t] * u[i, t])[:, None] * _wide(p["B"][i, t], D))
            pre[i, t] = (h[i, t + 1] * _wide(p["C"][i, t], D)).sum(1)
            if p["D"] is not None:
                pre[i, t] += p["D"] * u[i, t]
    y = pre if p["z"] is None else pre * silu(p["z"].astype(np.float64))
    for i in range(B):
        y[i, lens[i]:] = 0
    return y, h, pre, dt, raw


def scan_bwd(p, lens, dy, dh):
    y, h, pre, dt, raw = scan(p, lens)
    u, A = p["u"].astype(np.float64), p["A"].astype(np.float64)
    B, T, D = u.shape
    G, N = p["B"].shape[2:]
    skip = np.zeros(D) if p["D"] is None else p["D"].astype(np.float64)
    g = dict(du=np.zeros_like(u), ddelta=np.zeros_like(u), dA=np.zeros_like(A), dB=np.zeros((B, T, G, N)),
             dC=np.zeros((B, T, G, N)), dD=np.zeros(D), dz=np.zeros_like(u), ddelta_bias=np.zeros(D),
             dh0=np.zeros((B, D, N)))
    for i in range(B):
        gh = np.zeros((D, N)) if dh is None else dh[i].astype(np.float64)
        for t in reversed(range(lens[i])):
            d = dy[i, t].astype(np.float64)
            yb = d if p["z"] is None else d * silu(p["z"][i, t].astype(np.float64))
            if p["z"] is not None:
                g["dz"][i, t] = d * pre[i, t] * dsilu(p["z"][i, t].astype(np.float64))
            gh = gh + yb[:, None] * _wide(p["C"][i, t], D)
            g["dC"][i, t] = (yb[:, None] * h[i, t + 1]).reshape(G, D // G, N).sum(1)
            g["dB"][i, t] = (gh * (dt[i, t] * u[i, t])[:, None]).reshape(G, D // G, N).sum(1)
            q = (gh * _wide(p["B"][i, t], D)).sum(1)
            gh = gh * np.exp(dt[i, t][:, None] * A)
            w = gh * h[i, t]
            ddt = (w * A).sum(1) + u[i, t] * q
            g["dA"] += w * dt[i, t][:, None]
            g["du"][i, t] = dt[i, t] * q + skip * yb
            g["ddelta"][i, t] = ddt * (sigmoid(raw[i, t]) if p["softplus"] else 1.0)
            g["dD"] += yb * u[i, t]
            g["ddelta_bias"] += g["ddelta"][i, t]
        g["dh0"][i] = gh
    return g


# ---- error bounds of fp32 arithmetic ----
# U is half a step of fp32.  The exponential and the quotient of the fast functions are off by
# at most 2 steps each (2 x 2U) plus, for e^x, the rounding of its scaled exponent (|x| log2 e U
# absolute, so that much relative); E(x) = (4 + 2 |x|) U covers the exponential, and sigmoid, silu
# and their derivatives are within S(x) = (16 + 4 |x|) U of their own magnitude bound.
U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


def e_exp(x):
    return (4 + 2 * np.abs(x)) * U


def e_sig(x):
    return (16 + 4 * np.abs(x)) * U


def conv_bounds(x, w, b, state, lens, act, dtype, dy=None, dlast=None):
    """Absolute error bounds of y and, given dy, of dx, dw, db, dstate."""
    B, T, C = x.shape
    W = w.shape[1]
    ab = lambda v: None if v is None else np.abs(v)  # noqa: E731
    _, mag, _ = conv(np.abs(x), np.abs(w), ab(b), ab(state), lens, False)
    y, p, _ = conv(x, w, b, state, lens, act)
    ep = (W + 1) * U * mag
    # |silu'| <= 1.1
    ey = HALF[dtype] * np.abs(y) + ((1.1 * ep + e_sig(p) * np.abs(p)) if act else ep)
    if dy is None:
        return ey
    dp = np.abs(dy) * np.where(act, 1.1, 1.0)
    edp = np.abs(dy) * (0.5 * ep + e_sig(p)) if act else np.zeros_like(dp)   # |silu''| <= 1/2
    dx, _, _, dst = conv_bwd(x, w, b, state, lens, act, dy, dlast)
    n = sum(lens)
    mx, mw, mb, ms = conv_bwd(np.abs(x), np.abs(w), b, ab(state), lens, False, dp, ab(dlast))
    xx, xw, xb, xs = conv_bwd(np.abs(x), np.abs(w), b, ab(state), lens, False, edp, None)
    return (ey, xx + (W + 1) * U * mx + HALF[dtype] * np.abs(dx), xw + n * U * mw, xb + n * U * mb,
            xs + (W + 1) * U * ms + HALF[dtype] * np.abs(dst))


def scan_bounds(p, lens, dtype, dy=None, dh=None):
    """Absolute error bounds of the scan's outputs: y, h_final and, given dy, the gradients.
    Every quantity's bound follows the recurrence that makes it: the decays' relative error
    (the exponential's, and its argument's: dt's relative error and two roundings), the
    products' and sums' roundings, and the errors of what enters.  Doubled at the end: segments
    compose the same decays in another order, which rounds each of them once more."""
    y, h, pre, dt, raw = scan(p, lens)
    u, A = p["u"].astype(np.float64), p["A"].astype(np.float64)
    B, T, D = u.shape
    G, N = p["B"].shape[2:]
    skip = np.zeros(D) if p["D"] is None else np.abs(p["D"].astype(np.float64))
    out = HALF[dtype]
    # softplus: its exponential's relative error is its own (log(1 + e) moves by at most e's
    # share), and a dozen roundings of the series; the sum delta + bias rounds absolutely
    edt = ((12 + 2 * np.abs(raw)) * U + np.abs(raw) * U) if p["softplus"] else U * np.ones_like(raw)
    z = None if p["z"] is None else p["z"].astype(np.float64)
    sz = np.ones_like(u) if z is None else np.abs(silu(z))
    esz = np.zeros_like(u) if z is None else e_sig(z)     # relative to |z|, which is >= |silu|
    zm = np.ones_like(u) if z is None else np.maximum(np.abs(z), 1e-300)
    Eh = np.zeros((B, T + 1, D, N))
    Epre = np.zeros((B, T, D))
    dec, ea = np.zeros((B, T, D, N)), np.zeros((B, T, D, N))
    for i in range(B):
        for t in range(T):
            if t >= lens[i]:
                Eh[i, t + 1] = Eh[i, t]
                continue
            x = dt[i, t][:, None] * A
            dec[i, t] = np.exp(x)
            ea[i, t] = e_exp(x) + np.abs(x) * (edt[i, t][:, None] + 2 * U)
            add = np.abs(dt[i, t] * u[i, t])[:, None] * np.abs(_wide(p["B"][i, t], D))
            Eh[i, t + 1] = (dec[i, t] * Eh[i, t] + np.abs(dec[i, t] * h[i, t]) * ea[i, t]
                            + add * (edt[i, t][:, None] + 3 * U) + U * np.abs(h[i, t + 1]))
            Cw = np.abs(_wide(p["C"][i, t], D))
            mag = (Cw * np.abs(h[i, t + 1])).sum(1) + skip * np.abs(u[i, t])
            Epre[i, t] = (Cw * Eh[i, t + 1]).sum(1) + (N + 3) * U * mag
    Ey = Epre * sz + np.abs(pre) * zm * esz + out * np.abs(y)
    bounds = dict(y=2 * Ey, h=2 * Eh[:, -1] + 1e-30)
    if dy is None:
        return bounds
    g = scan_bwd(p, lens, dy, dh)
    z0 = lambda *s: np.zeros(s)  # noqa: E731
    e = dict(du=z0(B, T, D), ddelta=z0(B, T, D), dA=z0(D, N), dB=z0(B, T, G, N), dC=z0(B, T, G, N), dD=z0(D),
             dz=z0(B, T, D), ddelta_bias=z0(D), dh0=z0(B, D, N))
    per, n = D // G, sum(lens)
    for i in range(B):
        gh = z0(D, N) if dh is None else dh[i].astype(np.float64)
        Eg = z0(D, N)
        for t in reversed(range(lens[i])):
            d = np.abs(dy[i, t].astype(np.float64))
            sg = 1.0 if z is None else silu(z[i, t])
            yb, Eyb = dy[i, t] * sg, d * zm[i, t] * esz[i, t] + U * d * sz[i, t]
            if z is not None:
                e["dz"][i, t] = d * 1.1 * Epre[i, t] + d * np.abs(pre[i, t]) * (esz[i, t] + 2 * U)
            Bw, Cw = _wide(p["B"][i, t], D), _wide(p["C"][i, t], D)
            add = yb[:, None] * Cw
            gh = gh + add
            Eg = Eg + np.abs(Cw) * Eyb[:, None] + U * (np.abs(add) + np.abs(gh))
            ayb, ah = np.abs(yb)[:, None], np.abs(h[i, t + 1])
            fold = lambda m: m.reshape(G, per, N).sum(1)  # noqa: E731
            e["dC"][i, t] = fold(ayb * Eh[i, t + 1] + ah * Eyb[:, None] + (per + 2) * U * ayb * ah)
            du = (dt[i, t] * u[i, t])[:, None]
            e["dB"][i, t] = fold(np.abs(du) * Eg + np.abs(gh * du) * (edt[i, t][:, None] + (per + 3) * U))
            q = (gh * Bw).sum(1)
            Eq = (np.abs(Bw) * Eg).sum(1) + (N + 1) * U * np.abs(gh * Bw).sum(1)
            Eg = dec[i, t] * Eg + np.abs(dec[i, t] * gh) * (ea[i, t] + U)
            gh = gh * dec[i, t]
            w = gh * h[i, t]
            Ew = np.abs(h[i, t]) * Eg + np.abs(gh) * Eh[i, t] + U * np.abs(w)
            ddt = (w * A).sum(1) + u[i, t] * q
            Eddt = ((np.abs(A) * Ew).sum(1) + (N + 4) * U * np.abs(w * A).sum(1)
                    + np.abs(u[i, t]) * Eq + 2 * U * np.abs(u[i, t] * q))
            sig = sigmoid(raw[i, t]) if p["softplus"] else 1.0
            es = e_sig(raw[i, t]) if p["softplus"] else 0.0
            e["ddelta"][i, t] = Eddt * sig + np.abs(ddt) * es
            e["dA"] += dt[i, t][:, None] * Ew + np.abs(dt[i, t][:, None] * w) * (edt[i, t][:, None] + (n + 2) * U)
            e["du"][i, t] = (np.abs(dt[i, t]) * Eq + np.abs(dt[i, t] * q) * (edt[i, t] + 2 * U) + skip * Eyb
                             + 2 * U * skip * np.abs(yb))
            e["dD"] += np.abs(u[i, t]) * Eyb + (n + 1) * U * np.abs(yb * u[i, t])
            e["ddelta_bias"] += e["ddelta"][i, t] + n * U * np.abs(g["ddelta"][i, t])
        e["dh0"][i] = Eg
    for k in e:
        stored = out if k in ("du", "ddelta", "dz", "dB", "dC") else U
        bounds[k] = 2 * e[k] + stored * np.abs(g[k]) + 1e-30
    return bounds, g
