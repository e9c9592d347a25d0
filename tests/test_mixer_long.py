"""The operators around a token mixer at sizes where a block walks many rows, a run holds many
tokens and a sequence many segments, against the 64-bit definitions.  What smaller sizes leave
out: a norm block's second and later rows (rows on their way, alternating sums), the
convolution's bodies without tests of the edges, and the scan cut into segments."""
import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from tests import _mixer_ref as ref
from tests import _mixer_vec as vec
from tests.test_mixer_parity import (conv_inputs, dev, host, norm_inputs, norm_tol, rounded, same, scan_inputs,
                                     scan_tensors, within)

pytestmark = pytest.mark.gpu
U = ref.U


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_chunkwise_gb300 import build
    build.build()
    ldn.load()


# ---- RMS norm: three rows a block and more, in a number that is no multiple of the blocks ----
# blocks forward: 152 x max(1, 768 / threads), gradient: 152 x max(1, 512 / threads), one an SM past
# 8192 channels; threads: channels / 8 (or / 16, / 32, / 64 from 4096, 8193, 16385 on) in whole warps
ROWS = [(9500, 64), (4000, 777), (1500, 2048), (1400, 4096), (1100, 5001), (700, 8192), (1000, 9001), (700, 20000)]


@pytest.mark.parametrize("rows,D", ROWS)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", None)])
def test_add_rmsnorm_of_many_rows(rows, D, dtype, res):
    import torch
    x, r, w = norm_inputs(rows, D, dtype, res or dtype, seed=rows)
    gx, gr, gw = dev(x, dtype), dev(r, res) if res else None, dev(w)
    y, s = ldn.add_rmsnorm(gx, gr, gw, eps=1e-5)
    if res:
        assert torch.equal(s, (gx.float() + gr.float()).to(gr.dtype))
    want = ref.norm(host(s), w, 1e-5)
    within(y, want, norm_tol(want, dtype, D), "y")
    if res:     # in place
        again, s2 = ldn.add_rmsnorm(gx, gr, gw, eps=1e-5, residual_out=gr)
        assert s2 is gr and torch.equal(s, s2) and torch.equal(y, again)


@pytest.mark.parametrize("rows,D", ROWS)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_add_rmsnorm_e4m3_of_many_rows(rows, D, group, dtype):
    x, r, w = norm_inputs(rows, D, dtype, dtype, seed=rows + 1)
    q, scale, s = ldn.add_rmsnorm_e4m3(dev(x, dtype), dev(r, dtype), dev(w), eps=1e-5, group=group)
    want = ref.norm(host(s), w, 1e-5)
    sc = ref.groups_of(want, group)
    rel = (28 + D / 256) * U
    within(host(scale).reshape(rows, -1), sc, sc * rel, "scale")
    v = want / np.repeat(sc, group or D, axis=1)[:, :D]
    within(q, v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + np.abs(v) * 2 * rel, "q")


@pytest.mark.parametrize("rows,D", ROWS)
@pytest.mark.parametrize("dtype,res,add", [("bf16", "bf16", False), ("bf16", "f32", True), ("f32", "f32", True)])
def test_add_rmsnorm_backward_of_many_rows(rows, D, dtype, res, add):
    import torch
    r = np.random.default_rng(rows + 2)
    s, dy = rounded(2 * r.normal(size=(rows, D)), res), rounded(r.normal(size=(rows, D)), dtype)
    dsum = rounded(r.normal(size=(rows, D)), res) if add else None
    w = rounded(1 + 0.1 * r.normal(size=D), "f32")
    args = (dev(dy, dtype), dev(s, res), dev(w), dev(dsum, res))
    g = ldn.add_rmsnorm_backward(*args, eps=1e-5)
    ds, dw = ref.norm_bwd(dy, s, w, dsum, 1e-5)
    rr = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-5)
    wd, sums = np.abs(w * dy), (24 + D / 128) * U
    mag = rr * (wd + np.abs(s) * rr * rr * (wd * np.abs(s)).mean(-1, keepdims=True)) * 2 * sums
    mag += 2 * U * (0 if dsum is None else np.abs(dsum))
    within(g["dx"], ds, mag + ref.HALF[dtype] * np.abs(ds) + 1e-30, "dx")
    within(g["dresidual"], ds, mag + ref.HALF[res] * np.abs(ds) + 1e-30, "dresidual")
    within(g["dweight"], dw, np.abs(dy * s * rr).sum(0) * (sums + (8 + rows / 8) * U) + 1e-30, "dweight")
    again = ldn.add_rmsnorm_backward(*args, eps=1e-5)
    assert all(torch.equal(g[k], again[k]) for k in g)


# ---- convolution: long runs ----
RUNS = [  # B, T, C, W, dtype, bias, act, pad
    (300, 150, 8, 4, "bf16", True, True, 0),
    (300, 151, 8, 4, "f32", True, True, 8),
    (300, 150, 5, 2, "bf16", False, True, 3),
    (300, 97, 12, 1, "bf16", True, True, 0),
    (300, 130, 8, 8, "bf16", True, True, 0),
    (300, 130, 7, 6, "f32", False, False, 0),
    (24, 200, 1100, 4, "bf16", True, True, 1100),
    (24, 200, 1100, 7, "bf16", True, True, 0),
    (24, 200, 1001, 3, "f32", True, True, 0),
]


@pytest.mark.parametrize("case", RUNS, ids=str)
def test_short_conv_and_backward_in_long_runs(case):
    import torch
    B, T, C, W, dtype, bias, act, pad = case
    aligned = C % 4 == 0
    fwd = vec.conv_run(B * -(-C // 512), T, W, 1, 4 if W > 4 else 7 if aligned else 5)
    bwd = vec.conv_run(B * -(-C // 128), T, W, 4, 2 if W > 4 else 4)
    # bodies without tests of the edges: whole batches of 4 (two together, and a batch ahead) and of 3
    assert fwd >= 13 and bwd >= W - 1 + 6
    p = conv_inputs(B, T, C, W, dtype, True, bias, seed=B + W)
    r = np.random.default_rng(1)
    n = [int(v) for v in r.integers(0, T + 1, size=B)]
    n[0], n[1], n[2] = T, 0, 1
    x = p["x"].copy()
    dy, dl = rounded(r.normal(size=(B, T, C)), dtype), rounded(r.normal(size=(B, W - 1, C)), dtype)
    dyn = dy.copy()
    for i in range(B):
        x[i, n[i]:] = dyn[i, n[i]:] = np.nan            # rows past the end are not read
    gx, gl = dev(x, dtype, pad=pad, off=pad), dev(np.array(n))
    gw, gb, gs = dev(p["w"]), dev(p["b"]), dev(p["state"], dtype)
    args = (p["x"], p["w"], p["b"], p["state"], n, act)
    y, last = ldn.short_conv(gx, gw, gb, gs, lens=gl, activation=act)
    want, _, wlast = vec.conv(*args)
    ey, edx, edw, edb, eds = vec.conv_bounds(*args, dtype, dy, dl)
    within(y, want, ey + 1e-30, "y")
    assert np.array_equal(host(last), wlast)
    g = ldn.short_conv_backward(gx, gw, gb, dev(dyn, dtype), gs, dev(dl, dtype), lens=gl, activation=act)
    dx, dw, db, dst = vec.conv_bwd(*args, dy, dl)
    within(g["dx"], dx, edx + 1e-30, "dx")
    within(g["dweight"], dw, edw + 1e-30, "dweight")
    if bias:
        within(g["dbias"], db, edb + 1e-30, "dbias")
    within(g["dstate"], dst, eds + 1e-30, "dstate")
    again = ldn.short_conv_backward(gx, gw, gb, dev(dyn, dtype), gs, dev(dl, dtype), lens=gl, activation=act)
    assert all(g[k] is None or torch.equal(g[k], again[k]) for k in g)
    # whole sequences without a state: no run but the last has an edge
    y, _ = ldn.short_conv(dev(p["x"], dtype), gw, gb, None, activation=act)
    args = (p["x"], p["w"], p["b"], None, [T] * B, act)
    ey = vec.conv_bounds(*args, dtype, dy, None)[0]
    within(y, vec.conv(*args)[0], ey + 1e-30, "y of whole sequences")


# ---- scan: segments ----
SEGMENTS = [  # B, T, D, N, G, dtype, options, lens, pad, off
    (1, 545, 20, 16, 1, "bf16", {}, None, 0, 0),
    (2, 700, 6, 32, 2, "f32", {}, [700, 200], 0, 0),            # ends inside an early segment
    (3, 513, 24, 64, 1, "bf16", {}, [0, 513, 129], 8, 8),
    (3, 513, 24, 64, 1, "f32", dict(z=False), [512, 1, 513], 0, 0),
    (2, 1100, 12, 8, 3, "bf16", {}, [1100, 640], 3, 1),
    (2, 1100, 96, 8, 2, "f32", dict(skip=False), [1101, 161], 4, 4),
    (1, 2200, 5, 16, 5, "f32", {}, [1543], 0, 0),
    (1, 600, 40, 16, 1, "bf16", dict(z=False, skip=False, bias=False, h0=False), None, 0, 0),
    (2, 600, 72, 32, 3, "bf16", dict(softplus=False), [31, 600], 0, 0),
    (1, 8300, 2, 8, 1, "f32", {}, [8299], 0, 0),                 # 64 segments, the most there are
]
WHOLE = [  # gradients in segments of one part, and in no segments over many tiles; forward unsplit
    (1, 390, 100, 8, 100, "f32", {}, [390], 0, 0),
    (4, 390, 400, 32, 25, "f32", {}, [390, 0, 129, 300], 0, 0),
    (1, 300, 160, 16, 160, "bf16", {}, [299], 0, 0),
]


def long_memory(case):
    """A case's inputs with rates of a 64th, so that states reach over several segments."""
    B, T, D, N, G, dtype, opts = case[:7]
    p = scan_inputs(B, T, D, N, G, dtype, seed=T, **opts)
    p["A"] = p["A"] / 64
    return p


@pytest.mark.parametrize("case", SEGMENTS + WHOLE, ids=str)
def test_selective_scan_and_backward_in_segments(case):
    import torch
    B, T, D, N, G, dtype, opts, lens, pad, off = case
    assert (ldn.ldn_ssm_scan_workspace_size(B, T, D, N, G) > 0) == (case in SEGMENTS)
    p = long_memory(case)
    n = [T] * B if lens is None else [min(max(v, 0), T) for v in lens]
    t, sp = scan_tensors(p, n, dtype, pad, off), p["softplus"]
    gl, h0 = dev(None if lens is None else np.array(lens)), dev(p["h0"])
    r = np.random.default_rng(8)
    dy, dh = rounded(r.normal(size=(B, T, D)), dtype), rounded(r.normal(size=(B, D, N)), "f32")
    bound, grads = ref.scan_bounds(p, n, dtype, dy, dh)
    wy = ref.scan(p, n)[0]
    wh, eh = vec.state_bounds(p, n)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    outs = {}
    for what, ws in (("segments", None), ("unsplit", none)):
        y, h, states = outs[what] = ldn.selective_scan(*t, h0, delta_softplus=sp, lens=gl, save_states=True,
                                                       workspace=ws)
        within(y, wy, bound["y"] + 1e-30, f"y, {what}")
        within(h, wh[:, -1], bound["h"], f"h_final, {what}")
        within(states, wh[:, :-1:32], eh[:, :-1:32], f"states, {what}")
        again = ldn.selective_scan(*t, h0, delta_softplus=sp, lens=gl, workspace=ws)
        assert torch.equal(again[0], y) and torch.equal(again[1], h)
    if case in SEGMENTS:    # two ways of the same sums: not the same roundings everywhere
        assert not all(torch.equal(a, b) for a, b in zip(*outs.values()))
    dyn = dy.copy()
    for i in range(B):
        dyn[i, n[i]:] = np.nan
    args = (*t, outs["segments"][2], dev(dyn, dtype), dev(dh))
    g = ldn.selective_scan_backward(*args, delta_softplus=sp, lens=gl)
    for k, want in grads.items():
        given = dict(dD=p["D"], dz=p["z"], ddelta_bias=p["bias"]).get(k, 0)
        if given is None:
            assert g[k] is None
        else:
            within(g[k], want, bound[k], k)
    again = ldn.selective_scan_backward(*args, delta_softplus=sp, lens=gl)
    assert all(g[k] is None or torch.equal(g[k], again[k]) for k in g)


def test_segments_on_streams_and_in_graphs():
    """A scan in segments and its gradient, interleaved on two streams and replayed from two graphs
    at once: each call has a workspace of its own, and the bits are the same."""
    import torch
    p = long_memory((1, 1300, 24, 16, 1, "bf16", {}))
    t, h0 = scan_tensors(p, [1300], "bf16"), dev(p["h0"])
    assert ldn.ldn_ssm_scan_workspace_size(1, 1300, 24, 16, 1) > 0
    dy = dev(np.random.default_rng(1).normal(size=(1, 1300, 24)), "bf16")
    states = ldn.selective_scan(*t, h0, save_states=True)[2]
    for f in (lambda **k: ldn.selective_scan(*t, h0, save_states=True, **k),
              lambda **k: tuple(ldn.selective_scan_backward(*t, states, dy, h0, **k).values())):
        want = f()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = [f(stream=s) for _ in range(4) for s in (s1, s2)]
        torch.cuda.synchronize()
        assert all(same(want, g) for g in got)
        graphs, outs = [], []
        for s in (s1, s2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(f(stream=s))
            graphs.append(g)
        for _ in range(3):
            for g, s in zip(graphs, (s1, s2)):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(same(want, o) for o in outs)


def test_infinite_rates_and_steps_over_segments():
    """Rates of -infinity among ordinary ones in a scan of segments and in its gradient (a rate of
    -1e30 in 64 bits is one that forgets as well); a step of -infinity (a masked token) keeps the
    state, NaN stays in its channel; one sequence ends in an early segment."""
    import torch
    case = (2, 700, 8, 16, 1, "f32", {})
    p, n = long_memory(case), [700, 350]
    p["A"][3], p["A"][5, 2] = -1e30, -1e30
    assert ldn.ldn_ssm_scan_workspace_size(*case[:5]) > 0
    t, gl, h0 = scan_tensors(p, n, "f32"), dev(np.array(n)), dev(p["h0"])
    t[2][3], t[2][5, 2] = -float("inf"), -float("inf")
    r = np.random.default_rng(8)
    dy, dh = rounded(r.normal(size=(2, 700, 8)), "f32"), rounded(r.normal(size=(2, 8, 16)), "f32")
    bound, grads = ref.scan_bounds(p, n, "f32", dy, dh)
    wh, eh = vec.state_bounds(p, n)
    y, h, states = ldn.selective_scan(*t, h0, lens=gl, save_states=True)
    within(y, ref.scan(p, n)[0], bound["y"] + 1e-30, "y")
    within(h, wh[:, -1], bound["h"], "h_final")
    within(states, wh[:, :-1:32], eh[:, :-1:32], "states")
    g = ldn.selective_scan_backward(*t, states, dev(dy), dev(dh), lens=gl)
    for k, want in grads.items():
        within(g[k], want, bound[k], k)
    # masked tokens and NaN
    t[1][:, 40:700:3, 1] = -float("inf")
    t[0][0, 300, 6] = float("nan")
    q = dict(p, delta=p["delta"].copy())
    q["delta"][:, 40:700:3, 1] = -1e4        # a step of e^-10000 is zero in 64 bits as well
    y, h = ldn.selective_scan(*t, h0, lens=gl)
    keep = [c for c in range(8) if c != 6]
    bound, wh = ref.scan_bounds(q, n, "f32"), ref.scan(q, n)[1]
    within(h[:, keep], wh[:, -1][:, keep], bound["h"][:, keep], "h_final over masked tokens")
    assert torch.isnan(h[0, 6]).all() and torch.isfinite(h[1]).all() and torch.isnan(y[0, 300:, 6]).all()
    assert torch.isfinite(y[0, :300]).all() and torch.isfinite(y[1]).all() and torch.isfinite(y[0][:, keep]).all()
