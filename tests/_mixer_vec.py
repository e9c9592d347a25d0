"""The short convolution's reference and error bounds of tests/_mixer_ref.py over whole batches at
once, for sizes at which a loop over tokens takes too long, and the bound of every state of the
scan.  tests/test_mixer_edges_cpu.py compares them with the originals."""
import numpy as np

from tests._mixer_ref import HALF, U, _wide, dsilu, e_exp, e_sig, scan, silu


def _rows(x, state, lens, W):
    """The rows -(W-1) .. T-1, those past a sequence's end zero; whether a row is inside."""
    B, T, C = x.shape
    live = (np.arange(T) < np.asarray(lens)[:, None])[:, :, None]
    head = np.zeros((B, W - 1, C)) if state is None else state.astype(np.float64)
    return np.concatenate([head, np.where(live, x, 0)], 1).astype(np.float64), live


def conv(x, w, b, state, lens, act):
    T, W = x.shape[1], w.shape[1]
    rows, live = _rows(x, state, lens, W)
    p = sum(rows[:, j:j + T] * w[:, j] for j in range(W)) + (0 if b is None else b)
    p = np.where(live, p, 0)
    at = (np.asarray(lens)[:, None] + np.arange(W - 1))[:, :, None]
    return (silu(p) if act else p), p, np.take_along_axis(rows, at, 1)


def conv_bwd(x, w, b, state, lens, act, dy, dlast):
    B, T, C = x.shape
    W = w.shape[1]
    rows, live = _rows(x, state, lens, W)
    dp = np.where(live, dy, 0).astype(np.float64)
    if act:
        dp = dp * dsilu(conv(x, w, b, state, lens, act)[1])
    drows = np.zeros_like(rows)
    dw = np.zeros((C, W))
    for j in range(W):
        drows[:, j:j + T] += dp * w[:, j]
        dw[:, j] = (dp * rows[:, j:j + T]).sum((0, 1))
    if dlast is not None:
        for i in range(B):
            drows[i, lens[i]:lens[i] + W - 1] += dlast[i]
    return drows[:, W - 1:], dw, dp.sum((0, 1)), drows[:, :W - 1]


def conv_bounds(x, w, b, state, lens, act, dtype, dy, dlast):
    W = w.shape[1]
    ab = lambda v: None if v is None else np.abs(v)  # noqa: E731
    mag = conv(np.abs(x), np.abs(w), ab(b), ab(state), lens, False)[0]
    y, p, _ = conv(x, w, b, state, lens, act)
    ep = (W + 1) * U * mag
    ey = HALF[dtype] * np.abs(y) + ((1.1 * ep + e_sig(p) * np.abs(p)) if act else ep)
    dp = np.abs(dy) * (1.1 if act else 1.0)
    edp = np.abs(dy) * (0.5 * ep + e_sig(p)) if act else np.zeros_like(dp)
    dx, _, _, dst = conv_bwd(x, w, b, state, lens, act, dy, dlast)
    n = sum(lens)
    mx, mw, mb, ms = conv_bwd(np.abs(x), np.abs(w), b, ab(state), lens, False, dp, ab(dlast))
    xx, xw, xb, xs = conv_bwd(np.abs(x), np.abs(w), b, ab(state), lens, False, edp, None)
    return (ey, xx + (W + 1) * U * mx + HALF[dtype] * np.abs(dx), xw + n * U * mw, xb + n * U * mb,
            xs + (W + 1) * U * ms + HALF[dtype] * np.abs(dst))


def conv_run(units, T, W, per, blocks_sm):
    """Tokens of a run, as the kernels' launch cuts them."""
    fit, best, least = 152 * blocks_sm, 8, None
    for w in range(1, 5):
        rb = max(1, w * fit // max(1, units))
        run = max(8, -(-T // (rb * per)))
        runs = -(-T // run)
        cost = -(-units * -(-runs // per) // fit) * (run + W - 1 + 8)
        if least is None or cost < least:
            best, least = run, cost
    return best


def state_bounds(p, lens):
    """Every state [B][T+1][D][N] of the scan and the bound of its error: the recurrence of
    tests/_mixer_ref.py's scan_bounds, doubled as there."""
    _, h, _, dt, raw = scan(p, lens)
    u, A = p["u"].astype(np.float64), p["A"].astype(np.float64)
    T, D = u.shape[1:]
    edt = ((12 + 2 * np.abs(raw)) * U + np.abs(raw) * U) if p["softplus"] else U * np.ones_like(raw)
    E = np.zeros_like(h)
    for i in range(u.shape[0]):
        for t in range(T):
            if t >= lens[i]:
                E[i, t + 1] = E[i, t]
                continue
            x = dt[i, t][:, None] * A
            ea = e_exp(x) + np.abs(x) * (edt[i, t][:, None] + 2 * U)
            add = np.abs(dt[i, t] * u[i, t])[:, None] * np.abs(_wide(p["B"][i, t], D))
            E[i, t + 1] = (np.exp(x) * (E[i, t] + np.abs(h[i, t]) * ea) + add * (edt[i, t][:, None] + 3 * U)
                           + U * np.abs(h[i, t + 1]))
    return h, 2 * E + 1e-30
