"""The operators around a token mixer on the GPU against their 64-bit definitions.

Tolerances are absolute bounds worked out for every value from the arithmetic that makes it
(tests/_mixer_ref.py): half a step of the stored type, and fp32 roundings followed through the
recurrences."""
import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from tests import _mixer_ref as ref

pytestmark = pytest.mark.gpu
U = ref.U


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_chunkwise_gb300 import build
    build.build()
    ldn.load()


def _t(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def dev(a, dtype="f32", *, pad=0, off=0):
    """A GPU copy of an array.  pad: as a slice of rows that are `pad` elements wider, `off`
    elements in."""
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    t = t.to(_t(dtype)) if t.is_floating_point() else t.to(torch.int32)
    if pad:
        wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        wide[..., off:off + t.shape[-1]] = t
        return wide[..., off:off + t.shape[-1]]
    if off:
        flat = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
        flat[off:] = t.reshape(-1)
        return flat[off:].reshape(t.shape)
    return t


def host(t):
    return t.detach().double().cpu().numpy()


def rounded(a, dtype):
    """The values of an array once stored in dtype."""
    return None if a is None else host(dev(a, dtype))


def within(got, want, bound, what=""):
    got = host(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), what
    over = np.abs(got - want) - bound
    assert over.size == 0 or over.max() <= 0, f"{what}: {over.max():.3g} over the bound at {np.argmax(over)}"


# ---- RMS norm with the residual's addition ----
NORM_SIZES = [(1, 1), (3, 7), (2, 8), (5, 129), (1, 1000), (64, 2048), (3, 4095), (2, 4096), (7, 9001), (2, 32768)]


def norm_inputs(rows, D, dtype, res, seed=0):
    r = np.random.default_rng(seed)
    x = rounded(r.normal(size=(rows, D)), dtype)
    res_ = rounded(r.normal(size=(rows, D)) * 2, res)
    return x, res_, rounded(1 + 0.1 * r.normal(size=D), "f32")


def norm_tol(y, dtype, D):
    # the sum of squares: D / 32 additions a lane chain and a tree, halved by the root; the rest a few
    return np.abs(y) * (ref.HALF[dtype] + (24 + D / 256) * U) + 1e-30


@pytest.mark.parametrize("rows,D", NORM_SIZES)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", None), ("f32", None)])
def test_add_rmsnorm(rows, D, dtype, res):
    import torch
    x, r, w = norm_inputs(rows, D, dtype, res or dtype)
    gx, gr = dev(x, dtype), dev(r, res) if res else None
    y, s = ldn.add_rmsnorm(gx, gr, dev(w), eps=1e-5)
    assert y.dtype == _t(dtype)
    if res:
        assert torch.equal(s, (gx.float() + gr.float()).to(_t(res)))    # one fp32 addition, one rounding
    else:
        assert s is gx
    want = ref.norm(host(s), w, 1e-5)
    within(y, want, norm_tol(want, dtype, D), "y")


@pytest.mark.parametrize("rows,D", NORM_SIZES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32"), ("bf16", None)])
def test_add_rmsnorm_e4m3(rows, D, group, dtype, res):
    x, r, w = norm_inputs(rows, D, dtype, res or dtype, seed=1)
    q, scale, s = ldn.add_rmsnorm_e4m3(dev(x, dtype), dev(r, res) if res else None, dev(w), eps=1e-5, group=group)
    want = ref.norm(host(s), w, 1e-5)
    sc = ref.groups_of(want, group)
    assert scale.shape == ((rows,) if group == 0 else (rows, -(-D // 128)))
    rel = (28 + D / 256) * U
    got_sc = host(scale).reshape(rows, -1)
    within(got_sc, sc, sc * rel, "scale")
    v = want / np.repeat(sc, group or D, axis=1)[:, :D]
    # half a step of e4m3: 2^-4 of the value, 2^-10 below the smallest normal number
    within(q, v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + np.abs(v) * 2 * rel, "q")


def test_add_rmsnorm_e4m3_zero_and_tiny_rows():
    import torch
    x = torch.zeros(4, 256, device="cuda")
    x[1, 3] = 1e-38
    x[2] = 2.0
    w = torch.ones(256, device="cuda")
    w[128:] = 0
    q, scale, _ = ldn.add_rmsnorm_e4m3(x, None, w, eps=0.0, group=128)
    # eps = 0: a row of zeros has 1 / sqrt(0) = inf, and 0 * inf is not a number
    assert torch.isnan(q[0].float()).all()
    assert scale[2, 1].item() == pytest.approx(2.0 ** -100 / 448, rel=1e-6) and (q[2, 128:].float() == 0).all()
    q, scale, _ = ldn.add_rmsnorm_e4m3(x, None, w, eps=1e-6, group=0)
    assert (q[0].float() == 0).all() and scale[0].item() == pytest.approx(2.0 ** -100 / 448, rel=1e-6)
    assert (q[2, :128].float() == 448).all()


def test_add_rmsnorm_nan_and_infinity_stay_in_their_row():
    import torch
    x = torch.randn(4, 300, device="cuda")
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    w = torch.ones(300, device="cuda")
    y, _ = ldn.add_rmsnorm(x, None, w)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 9]) and torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert (y[2, :9] == 0).all()
    q, _, _ = ldn.add_rmsnorm_e4m3(x, None, w, group=128)
    assert torch.isnan(q[1].float()).all() and torch.isfinite(q[0].float()).all()


@pytest.mark.parametrize("rows,D", NORM_SIZES + [(700, 257), (2000, 64)])
@pytest.mark.parametrize("dtype,res,add", [("bf16", "bf16", True), ("bf16", "f32", True), ("f32", "f32", False)])
def test_add_rmsnorm_backward(rows, D, dtype, res, add):
    import torch
    r = np.random.default_rng(2)
    s, dy = rounded(2 * r.normal(size=(rows, D)), res), rounded(r.normal(size=(rows, D)), dtype)
    dsum = rounded(r.normal(size=(rows, D)), res) if add else None
    w = rounded(1 + 0.1 * r.normal(size=D), "f32")
    g = ldn.add_rmsnorm_backward(dev(dy, dtype), dev(s, res), dev(w), dev(dsum, res), eps=1e-5)
    ds, dw = ref.norm_bwd(dy, s, w, dsum, 1e-5)
    rr = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-5)
    wd, sums = np.abs(w * dy), (24 + D / 128) * U
    mag = rr * (wd + np.abs(s) * rr * rr * (wd * np.abs(s)).mean(-1, keepdims=True)) * 2 * sums
    mag += 2 * U * (0 if dsum is None else np.abs(dsum))
    within(g["dx"], ds, mag + ref.HALF[dtype] * np.abs(ds) + 1e-30, "dx")
    within(g["dresidual"], ds, mag + ref.HALF[res] * np.abs(ds) + 1e-30, "dresidual")
    assert (g["dx"] is g["dresidual"]) == (dtype == res)
    within(g["dweight"], dw, np.abs(dy * s * rr).sum(0) * (sums + (8 + rows / 8) * U) + 1e-30, "dweight")
    again = ldn.add_rmsnorm_backward(dev(dy, dtype), dev(s, res), dev(w), dev(dsum, res), eps=1e-5)
    assert all(torch.equal(g[k], again[k]) for k in g)


def test_add_rmsnorm_in_place_unaligned_and_empty():
    import torch
    x, r, w = norm_inputs(9, 200, "bf16", "bf16", seed=3)
    y0, s0 = ldn.add_rmsnorm(dev(x, "bf16"), dev(r, "bf16"), dev(w))
    res = dev(r, "bf16")
    y1, s1 = ldn.add_rmsnorm(dev(x, "bf16"), res, dev(w), residual_out=res)
    assert s1 is res and torch.equal(s0, s1) and torch.equal(y0, y1)
    # the same rows at an address that is no multiple of 16 bytes: single elements, the same sums
    y2, s2 = ldn.add_rmsnorm(dev(x, "bf16", off=1), dev(r, "bf16"), dev(w))
    assert torch.equal(s0, s2) and torch.equal(y0, y2)
    y3, s3 = ldn.add_rmsnorm(torch.empty(0, 200, device="cuda"), None, dev(w))
    assert y3.shape == (0, 200)
    g = ldn.add_rmsnorm_backward(torch.empty(0, 200, device="cuda"), torch.empty(0, 200, device="cuda"), dev(w))
    assert (g["dweight"] == 0).all()
    xs = dev(x, "bf16").reshape(3, 3, 200)
    assert ldn.add_rmsnorm_e4m3(xs, None, dev(w), group=128)[1].shape == (3, 3, 2)


# ---- short convolution ----
def conv_inputs(B, T, C, W, dtype, state, bias, seed=0):
    r = np.random.default_rng(seed)
    return dict(x=rounded(r.normal(size=(B, T, C)), dtype), w=rounded(r.normal(size=(C, W)) * W ** -0.5, "f32"),
                b=rounded(0.1 * r.normal(size=C), "f32") if bias else None,
                state=rounded(r.normal(size=(B, W - 1, C)), dtype) if state else None)


CONV_CASES = [  # B, T, C, W, dtype, state, bias, act, lens, pad, off
    (1, 1, 1, 1, "f32", False, False, True, None, 0, 0),
    (1, 1, 8, 4, "bf16", True, True, True, None, 0, 0),
    (2, 3, 64, 4, "bf16", True, True, True, None, 64, 0),
    (2, 2, 24, 8, "f32", True, False, False, [1, 2], 0, 0),
    (3, 33, 7, 3, "bf16", False, True, True, [0, 33, 2], 0, 0),
    (2, 70, 260, 4, "f32", True, True, True, [70, 1], 4, 4),
    (2, 70, 260, 4, "bf16", True, True, True, [69, 0], 5, 3),
    (4, 129, 520, 2, "bf16", False, False, True, [129, 128, 64, 65], 8, 8),
    (1, 300, 100, 5, "bf16", True, True, False, None, 0, 1),
    (2, 64, 36, 6, "f32", True, True, True, [200, -3], 0, 0),     # clamped to 64 and 0
    (1, 257, 1024, 7, "bf16", True, True, True, [250], 0, 0),
    (40, 65, 48, 4, "bf16", True, True, True, list(range(26, 66)), 0, 0),
]


@pytest.mark.parametrize("case", CONV_CASES, ids=str)
def test_short_conv_and_backward(case):
    import torch
    B, T, C, W, dtype, state, bias, act, lens, pad, off = case
    p = conv_inputs(B, T, C, W, dtype, state, bias)
    n = [T] * B if lens is None else [min(max(v, 0), T) for v in lens]
    x = p["x"].copy()
    for i in range(B):
        x[i, n[i]:] = np.nan            # rows past the end are not read
    gx, glens = dev(x, dtype, pad=pad, off=off), dev(None if lens is None else np.array(lens))
    gw, gb, gs = dev(p["w"]), dev(p["b"]), dev(p["state"], dtype)
    y, last = ldn.short_conv(gx, gw, gb, gs, lens=glens, activation=act)
    want, _, wlast = ref.conv(p["x"], p["w"], p["b"], p["state"], n, act)
    r = np.random.default_rng(9)
    dy, dl = rounded(r.normal(size=(B, T, C)), dtype), rounded(r.normal(size=(B, W - 1, C)), dtype)
    ey, edx, edw, edb, eds = ref.conv_bounds(p["x"], p["w"], p["b"], p["state"], n, act, dtype, dy, dl)
    within(y, want, ey + 1e-30, "y")
    assert np.array_equal(host(last), wlast)            # rows are copied
    dyn = dy.copy()
    for i in range(B):
        dyn[i, n[i]:] = np.nan
    g = ldn.short_conv_backward(gx, gw, gb, dev(dyn, dtype), gs, dev(dl, dtype), lens=glens, activation=act)
    dx, dw, db, dst = ref.conv_bwd(p["x"], p["w"], p["b"], p["state"], n, act, dy, dl)
    within(g["dx"], dx, edx + 1e-30, "dx")
    within(g["dweight"], dw, edw + 1e-30, "dweight")
    if bias:
        within(g["dbias"], db, edb + 1e-30, "dbias")
    else:
        assert g["dbias"] is None
    if state:
        within(g["dstate"], dst, eds + 1e-30, "dstate")
    again = ldn.short_conv_backward(gx, gw, gb, dev(dyn, dtype), gs, dev(dl, dtype), lens=glens, activation=act)
    assert all(g[k] is None or torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,C,W", [(1, 1, 2), (3, 7, 3), (2, 64, 4), (65, 1032, 4), (2, 24, 8), (2, 5, 1)])
def test_short_conv_step_continues_a_prompt(dtype, B, C, W):
    """Tokens one by one from a prompt's state give the longer prompt's rows, bit for bit
    (the same sums in the same order); in place and not."""
    import torch
    T, more = 5, 4
    p = conv_inputs(B, T + more, C, W, dtype, True, True, seed=4)
    x, w, b, s0 = dev(p["x"], dtype, pad=3, off=2), dev(p["w"]), dev(p["b"]), dev(p["state"], dtype)
    whole, last = ldn.short_conv(x, w, b, s0)
    _, st = ldn.short_conv(x[:, :T].contiguous(), w, b, s0)
    for t in range(T, T + more):
        if t % 2:
            y = ldn.short_conv_step(x[:, t], w, b, st)
        else:
            new = torch.empty_like(st)
            y, st = ldn.short_conv_step(x[:, t], w, b, st, state_out=new), new
        assert torch.equal(y, whole[:, t])
    assert torch.equal(st, last)


def test_short_conv_state_in_place_and_no_tokens():
    import torch
    p = conv_inputs(3, 2, 40, 6, "bf16", True, True, seed=5)
    x, w, b = dev(p["x"], "bf16"), dev(p["w"]), dev(p["b"])
    y0, s0 = ldn.short_conv(x, w, b, dev(p["state"], "bf16"))
    st = dev(p["state"], "bf16")
    y1, s1 = ldn.short_conv(x, w, b, st, state_out=st)
    assert s1 is st and torch.equal(s0, s1) and torch.equal(y0, y1)
    y, s = ldn.short_conv(x[:, :0], w, b, st)
    assert y.shape == (3, 0, 40) and torch.equal(s, st)
    g = ldn.short_conv_backward(x[:, :0], w, b, y, st, s0)
    assert torch.equal(g["dstate"], s0) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


# ---- selective scan ----
def scan_inputs(B, T, D, N, G, dtype, *, z=True, skip=True, bias=True, softplus=True, h0=True, seed=0):
    r = np.random.default_rng(seed)
    f = lambda *s: rounded(r.normal(size=s), dtype)  # noqa: E731
    delta = f(B, T, D)
    shift = r.normal(size=D) - 2
    if not softplus:    # steps as given are positive: a negative one grows the state without bound
        delta, shift = rounded(np.abs(delta) * 0.1, dtype), np.abs(shift) * 0.1
    return dict(u=f(B, T, D), delta=delta, A=rounded(-np.exp(r.normal(size=(D, N))), "f32"), B=f(B, T, G, N),
                C=f(B, T, G, N), D=rounded(r.normal(size=D), "f32") if skip else None, z=f(B, T, D) if z else None,
                bias=rounded(shift, "f32") if bias else None,
                h0=rounded(r.normal(size=(B, D, N)), "f32") if h0 else None, softplus=softplus)


def scan_tensors(p, n, dtype, pad=0, off=0):
    """GPU tensors in the order of the calls; rows past a sequence's end hold NaN."""
    def rows(a):
        if a is None:
            return None
        a = a.copy()
        for i in range(a.shape[0]):
            a[i, n[i]:] = np.nan
        return a
    G, N = p["B"].shape[2:]
    flat = lambda a: rows(a).reshape(*a.shape[:2], G * N)  # noqa: E731
    Bm, Cm = (dev(flat(p[k]), dtype, pad=pad, off=off).unflatten(-1, (G, N)) for k in "BC")
    return [dev(rows(p["u"]), dtype), dev(rows(p["delta"]), dtype, off=off), dev(p["A"]), Bm, Cm, dev(p["D"]),
            dev(rows(p["z"]), dtype, pad=pad, off=off), dev(p["bias"])]


SCAN_CASES = [  # B, T, D, N, G, dtype, options, lens, pad, off
    (1, 1, 1, 8, 1, "f32", {}, None, 0, 0),
    (1, 1, 8, 16, 1, "bf16", {}, None, 0, 0),
    (2, 31, 16, 16, 1, "bf16", {}, None, 8, 8),
    (2, 32, 40, 16, 2, "bf16", dict(z=False), None, 0, 0),
    (2, 33, 72, 16, 1, "f32", dict(skip=False), None, 4, 4),
    (3, 65, 24, 32, 3, "bf16", dict(h0=False), [65, 0, 33], 3, 1),
    (2, 70, 17, 64, 1, "f32", dict(bias=False), [1, 70], 0, 0),
    (2, 64, 96, 8, 2, "bf16", dict(softplus=False), [64, 63], 8, 0),
    (1, 130, 5, 16, 5, "bf16", {}, [97], 0, 0),
    (2, 40, 130, 8, 1, "f32", dict(z=False, skip=False, bias=False, h0=False), [500, -1], 0, 0),
    (1, 290, 20, 16, 1, "bf16", {}, None, 0, 0),                # segments
    (2, 420, 6, 32, 2, "f32", {}, [420, 200], 0, 0),            # segments, one sequence ends early
    (3, 37, 40, 16, 2, "f32", {}, [37, 0, 5], 0, 0),            # groups of an odd number of 16-byte vectors
    (3, 70, 24, 32, 2, "f32", {}, [1, 70, 33], 0, 0),
    (2, 34, 12, 64, 3, "f32", {}, [34, 2], 0, 0),
    (2, 300, 56, 8, 7, "bf16", {}, [2, 300], 0, 0),
    (2, 300, 40, 16, 5, "bf16", {}, [130, 300], 0, 0),
]


@pytest.mark.parametrize("case", SCAN_CASES, ids=str)
def test_selective_scan_and_backward(case):
    import torch
    B, T, D, N, G, dtype, opts, lens, pad, off = case
    p = scan_inputs(B, T, D, N, G, dtype, **opts)
    n = [T] * B if lens is None else [min(max(v, 0), T) for v in lens]
    t, sp = scan_tensors(p, n, dtype, pad, off), p["softplus"]
    gl, h0 = dev(None if lens is None else np.array(lens)), dev(p["h0"])
    y, h, states = ldn.selective_scan(*t, h0, delta_softplus=sp, lens=gl, save_states=True)
    r = np.random.default_rng(8)
    dy, dh = rounded(r.normal(size=(B, T, D)), dtype), rounded(r.normal(size=(B, D, N)), "f32")
    bound, grads = ref.scan_bounds(p, n, dtype, dy, dh)
    wy, wh = ref.scan(p, n)[:2]
    within(y, wy, bound["y"] + 1e-30, "y")
    within(h, wh[:, -1], bound["h"], "h_final")
    within(states[:, 0], wh[:, 0], np.zeros_like(wh[:, 0]), "the entering state")
    unsplit = ldn.selective_scan(*t, h0, delta_softplus=sp, lens=gl,
                                 workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    within(unsplit[0], wy, bound["y"] + 1e-30, "y unsplit")
    within(unsplit[1], wh[:, -1], bound["h"], "h_final unsplit")
    dyn = dy.copy()
    for i in range(B):
        dyn[i, n[i]:] = np.nan
    args = (*t, states, dev(dyn, dtype), dev(dh))
    g = ldn.selective_scan_backward(*args, delta_softplus=sp, lens=gl)
    for k, want in grads.items():
        given = dict(dD=p["D"], dz=p["z"], ddelta_bias=p["bias"]).get(k, 0)
        if given is None:
            assert g[k] is None
        else:
            within(g[k], want, bound[k], k)
    again = ldn.selective_scan_backward(*args, delta_softplus=sp, lens=gl)
    assert all(g[k] is None or torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,D,N,G,opts", [(1, 1, 8, 1, {}), (3, 40, 16, 2, {}), (65, 24, 32, 3, dict(z=False)),
                                          (2, 130, 64, 1, dict(skip=False, bias=False)),
                                          (2, 7, 16, 1, dict(softplus=False))])
def test_selective_scan_step(dtype, B, D, N, G, opts):
    """Tokens one by one from a prompt's state, against the whole in 64 bits; in place and not."""
    import torch
    T, more = 6, 5
    p = scan_inputs(B, T + more, D, N, G, dtype, seed=3, **opts)
    n = [T + more] * B
    bound, wy = ref.scan_bounds(p, n, dtype), ref.scan(p, n)
    u, dl, A, Bm, Cm, Ds, z, b = scan_tensors(p, n, dtype, 5, 3)
    cut = lambda m: None if m is None else m[:, :T].contiguous()  # noqa: E731
    _, h = ldn.selective_scan(cut(u), cut(dl), A, cut(Bm), cut(Cm), Ds, cut(z), b, dev(p["h0"]),
                              delta_softplus=p["softplus"])
    for t in range(T, T + more):
        at = lambda m: None if m is None else m[:, t]  # noqa: E731
        args = (at(u), at(dl), A, at(Bm), at(Cm), Ds, at(z), b, h)
        if t % 2:
            y = ldn.selective_scan_step(*args, delta_softplus=p["softplus"])
        else:
            h2 = torch.empty_like(h)
            y = ldn.selective_scan_step(*args, delta_softplus=p["softplus"], h_out=h2)
            h = h2
        within(y, wy[0][:, t], bound["y"][:, t] + 1e-30, f"y {t}")
    within(h, wy[1][:, -1], bound["h"], "h")


def test_selective_scan_no_tokens():
    import torch
    p = scan_inputs(2, 1, 12, 16, 1, "f32")
    t = scan_tensors(p, [1, 1], "f32")
    cut = [m[:, :0] if m is not None and m.dim() > 2 else m for m in t]
    h0 = dev(p["h0"])
    y, h, states = ldn.selective_scan(*cut, h0, save_states=True)
    assert y.shape == (2, 0, 12) and torch.equal(h, h0) and states.shape == (2, 0, 12, 16)
    g = ldn.selective_scan_backward(*cut, states, y, h0)
    assert torch.equal(g["dh0"], h0) and all((g[k] == 0).all() for k in ("dA", "dD", "ddelta_bias"))


def test_selective_scan_steps_of_all_magnitudes():
    """softplus keeps its relative accuracy for small steps and is the identity for large ones;
    a decay of e^-inf forgets, one of e^0 keeps."""
    import torch
    D, N = 64, 16
    raw = np.linspace(-30, 60, D).astype(np.float32).astype(np.float64)
    p = scan_inputs(1, 3, D, N, 1, "f32", z=False, skip=False)
    p["delta"], p["bias"] = np.broadcast_to(raw, (1, 3, D)).copy(), None
    t = scan_tensors(p, [3], "f32")
    y, h = ldn.selective_scan(*t, dev(p["h0"]))
    bound = ref.scan_bounds(p, [3], "f32")
    wy, wh = ref.scan(p, [3])[:2]
    within(y, wy, bound["y"] + 1e-30, "y")
    within(h, wh[:, -1], bound["h"], "h")


def test_selective_scan_forgets_and_keeps_at_infinity():
    """A rate of -infinity leaves only the last token's input, whatever rows lie behind the
    sequence's end; a step of -infinity (a masked token) leaves the state; NaN stays in its
    channel."""
    import torch
    p = scan_inputs(2, 40, 8, 16, 1, "f32", z=False)
    p["A"][3] = -np.inf
    p["A"][5] = -3.4e38
    p["delta"][:, 7:9, 1] = -np.inf
    p["u"][0, 2, 6] = np.nan
    n = [40, 35]
    t = scan_tensors(p, n, "f32")
    gl, h0 = dev(np.array(n)), dev(p["h0"])
    for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
        y, h = ldn.selective_scan(*t, h0, lens=gl, workspace=ws)
        dt = ref.softplus(p["delta"] + p["bias"])
        for i in range(2):
            for c in (3, 5):
                last = dt[i, n[i] - 1, c] * p["u"][i, n[i] - 1, c] * p["B"][i, n[i] - 1, 0]
                within(h[i, c], last, np.abs(last) * 64 * U + 1e-30, "only the last input")
        assert torch.isnan(h[0, 6]).all() and torch.isnan(y[0, 2:, 6]).all() and torch.isfinite(y[0, :2]).all()
        keep = [c for c in range(8) if c != 6]
        assert torch.isfinite(h[:, keep]).all() and torch.isfinite(y[1]).all() and torch.isfinite(y[0][:, keep]).all()
    # up to the masked tokens and over them, the state is the same
    cut = lambda k: [m[:, :k].contiguous() if m is not None and m.dim() > 2 else m for m in t]  # noqa: E731
    before, over = ldn.selective_scan(*cut(7), h0)[1], ldn.selective_scan(*cut(9), h0)[1]
    assert torch.equal(before[:, 1], over[:, 1]) and not torch.equal(before[:, 0], over[:, 0])


# ---- streams, graphs, several calls ----
def mixer_calls():
    """One call of each operator with fixed inputs: name -> (call, outputs)."""
    import torch
    x, r, w = norm_inputs(40, 520, "bf16", "f32")
    gx, gr, gw = dev(x, "bf16"), dev(r), dev(w)
    c = conv_inputs(2, 70, 264, 4, "bf16", True, True)
    cx, cw, cb, cs = dev(c["x"], "bf16"), dev(c["w"]), dev(c["b"]), dev(c["state"], "bf16")
    p = scan_inputs(1, 420, 24, 16, 1, "bf16")
    t, h0 = scan_tensors(p, [420], "bf16"), dev(p["h0"])
    dy, dh = dev(rounded(np.random.default_rng(1).normal(size=(1, 420, 24)), "bf16"), "bf16"), h0 * 2
    states = ldn.selective_scan(*t, h0, save_states=True)[2]
    one = [m[:, 0] if m is not None and m.dim() > 2 else m for m in t]
    torch.cuda.synchronize()
    return {
        "add_rmsnorm": lambda **k: ldn.add_rmsnorm(gx, gr, gw, **k),
        "add_rmsnorm_e4m3": lambda **k: ldn.add_rmsnorm_e4m3(gx, gr, gw, group=128, **k),
        "add_rmsnorm_backward": lambda **k: tuple(ldn.add_rmsnorm_backward(gx, gr, gw, **k).values()),
        "short_conv": lambda **k: ldn.short_conv(cx, cw, cb, cs, **k),
        "short_conv_step": lambda **k: (ldn.short_conv_step(cx[:, 3], cw, cb, cs, state_out=torch.empty_like(cs), **k),),
        "short_conv_backward": lambda **k: tuple(ldn.short_conv_backward(cx, cw, cb, cx, cs, cs, **k).values()),
        "selective_scan": lambda **k: ldn.selective_scan(*t, h0, save_states=True, **k),
        "selective_scan_step": lambda **k: (ldn.selective_scan_step(*one, h0, h_out=torch.empty_like(h0), **k),),
        "selective_scan_backward": lambda **k: tuple(ldn.selective_scan_backward(*t, states, dy, dh, **k).values()),
    }


def same(a, b):
    import torch
    return all(torch.equal(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                           y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y) for x, y in zip(a, b))


def test_calls_on_another_stream_and_side_by_side():
    import torch
    calls = mixer_calls()
    for name, f in calls.items():
        want = f()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = [f(stream=s) for _ in range(3) for s in (s1, s2)]      # interleaved, own workspaces
        torch.cuda.synchronize()
        assert all(same(want, g) for g in got), name
        with torch.cuda.stream(s1):
            g = f()
        torch.cuda.synchronize()
        assert same(want, g), name


def test_calls_captured_and_replayed():
    """Every call replays in a graph, bit for bit, also two captured calls whose graphs are
    replayed on two streams at once."""
    import torch
    calls = mixer_calls()
    for name, f in calls.items():
        want = f()
        torch.cuda.synchronize()
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(f())
            graphs.append(g)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(3):
            for g, s in zip(graphs, (s1, s2)):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(same(want, o) for o in outs), name


def test_torch_layer_refuses():
    import torch
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(TypeError):
        ldn.add_rmsnorm(x.half(), None, w)
    with pytest.raises(TypeError):
        ldn.add_rmsnorm(x, None, w.bfloat16())
    with pytest.raises(ValueError):
        ldn.add_rmsnorm(x, x[:2], w)
    with pytest.raises(ValueError):
        ldn.add_rmsnorm(x.t(), None, torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        ldn.add_rmsnorm(x, None, w, residual_out=x.clone())
    with pytest.raises(ldn.LdnError):
        ldn.add_rmsnorm_e4m3(x, None, w, group=64, scale=torch.empty(4, 1, device="cuda"))
    with pytest.raises(ldn.LdnError):
        ldn.add_rmsnorm(x, None, w, out=x)
    with pytest.raises(ValueError):
        ldn.short_conv(x, torch.ones(64, 4, device="cuda"))
    with pytest.raises(ldn.LdnError):
        ldn.short_conv(x[None], torch.ones(64, 9, device="cuda"))
    with pytest.raises(ValueError):
        ldn.short_conv(x[None], torch.ones(64, 4, device="cuda"), lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        ldn.short_conv(x[None], torch.ones(64, 4, device="cuda"), lens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        ldn.short_conv(x[None], torch.ones(64, 4, device="cuda"), lens=torch.zeros(1, dtype=torch.int32))
    B = torch.zeros(1, 4, 1, 24, device="cuda")
    with pytest.raises(ldn.LdnError):
        ldn.selective_scan(x[None], x[None], torch.zeros(64, 24, device="cuda"), B, B)
    h = torch.zeros(1, 64, 16, device="cuda")
    B = torch.zeros(1, 4, 1, 16, device="cuda")
    with pytest.raises(ldn.LdnError):
        ldn.selective_scan(x[None], x[None], torch.zeros(64, 16, device="cuda"), B, B, h0=h, h_final=h)
    with pytest.raises(TypeError):
        ldn.add_rmsnorm_e4m3(x, None, w, group=128.0)
    with pytest.raises(TypeError):
        ldn.add_rmsnorm(x, None, w, eps="small")
    with pytest.raises(RuntimeError):
        ldn.short_conv(x[None], torch.ones(64, 4, device="cuda"), activation=torch.ones(2))
    with pytest.raises(ValueError):
        ldn.add_rmsnorm(x, None, w, stream=3)
    with pytest.raises(ValueError):     # B of one row for x's four
        ldn.selective_scan_step(x, x, torch.zeros(64, 16, device="cuda"), B[:, 0], None, None, None, None, h)
    with pytest.raises(ldn.LdnError):
        ldn.add_rmsnorm(x.half().float(), None, w, eps=float("nan"))


# ---- the operators together ----
def test_a_block_for_a_prompt_and_single_tokens():
    """Norm, input projection, convolution, projections to (delta, B, C), scan with its output
    gate, output projection, next norm: a prompt and then tokens one by one, fp32, against the
    whole sequence in 64 bits."""
    import torch
    r = np.random.default_rng(11)
    B, T, more, M, D, N, W, R = 2, 37, 3, 48, 64, 16, 4, 8
    f = lambda *s, k=1.0: torch.from_numpy(r.normal(size=s) * k).double().cuda()  # noqa: E731
    P = dict(nw=1 + f(M, k=0.1), win=f(2 * D, M, k=M ** -0.5), cw=f(D, W, k=0.5), cb=f(D, k=0.1),
             wx=f(R + 2 * N, D, k=D ** -0.5), wdt=f(D, R, k=R ** -0.5), A=-torch.exp(f(D, N, k=0.5)), Ds=1 + f(D, k=0.1),
             bias=f(D, k=0.5) - 3, wout=f(M, D, k=D ** -0.5))
    P = {k: v.float().double() for k, v in P.items()}
    hid, res = f(B, T + more, M).float().double(), f(B, T + more, M).float().double()

    def whole():
        n_ = lambda a: a.cpu().numpy()  # noqa: E731
        s = hid + res
        x = torch.from_numpy(ref.norm(n_(s), n_(P["nw"]), 1e-6)).cuda()
        xz = x @ P["win"].t()
        xc = torch.from_numpy(ref.conv(n_(xz[..., :D]), n_(P["cw"]), n_(P["cb"]), None, [T + more] * B, True)[0]).cuda()
        db = xc @ P["wx"].t()
        delta = db[..., :R] @ P["wdt"].t()
        p = dict(u=n_(xc), delta=n_(delta), A=n_(P["A"]), B=n_(db[..., None, R:R + N]), C=n_(db[..., None, R + N:]),
                 D=n_(P["Ds"]), z=n_(xz[..., D:]), bias=n_(P["bias"]), h0=None, softplus=True)
        y = torch.from_numpy(ref.scan(p, [T + more] * B)[0]).cuda()
        return ref.norm(n_(y @ P["wout"].t() + s), n_(P["nw"]), 1e-6)

    F = {k: v.float().contiguous() for k, v in P.items()}
    hf, rf = hid.float(), res.float()

    def prompt():
        x, s = ldn.add_rmsnorm(hf[:, :T].contiguous(), rf[:, :T].contiguous(), F["nw"])
        xz = x @ F["win"].t()
        xc, cst = ldn.short_conv(xz[..., :D], F["cw"], F["cb"])
        db = xc @ F["wx"].t()
        delta = db[..., :R] @ F["wdt"].t()
        y, h = ldn.selective_scan(xc, delta, F["A"], db[..., R:R + N].unflatten(-1, (1, N)),
                                  db[..., R + N:].unflatten(-1, (1, N)), F["Ds"], xz[..., D:], F["bias"])
        return ldn.add_rmsnorm(y @ F["wout"].t(), s, F["nw"])[0], cst, h

    def token(t, cst, h):
        x, s = ldn.add_rmsnorm(hf[:, t].contiguous(), rf[:, t].contiguous(), F["nw"])
        xz = x @ F["win"].t()
        xc = ldn.short_conv_step(xz[..., :D], F["cw"], F["cb"], cst)
        db = xc @ F["wx"].t()
        y = ldn.selective_scan_step(xc, db[..., :R] @ F["wdt"].t(), F["A"], db[..., R:R + N].unflatten(-1, (1, N)),
                                    db[..., R + N:].unflatten(-1, (1, N)), F["Ds"], xz[..., D:], F["bias"], h)
        return ldn.add_rmsnorm(y @ F["wout"].t(), s, F["nw"])[0]

    torch.backends.cuda.matmul.allow_tf32 = False
    want = whole()
    y, cst, h = prompt()
    got = [host(y)]
    for t in range(T, T + more):
        got.append(host(token(t, cst, h))[:, None])
    got = np.concatenate(got, 1)
    # Six stages in fp32; the longest sum of a stage is 64 terms and the scan's memory about 40
    # steps, so each adds at most ~ 100 roundings of its magnitude, and a stage's output is at
    # most a few times its input: 6 x 100 x 4 roundings of the largest magnitude
    assert np.abs(got - want).max() <= 2400 * U * np.abs(want).max()
