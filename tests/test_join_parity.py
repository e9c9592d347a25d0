"""The operators that join blocks on the GPU against their 64-bit definitions, with bounds worked
out for every value from the arithmetic that makes it (tests/_join_ref.py), and the calls that their
documentation allows: strides, addresses, streams, graphs, in place, no rows, what is not finite."""
import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from tests import _join_ref as ref
from tests.test_mixer_parity import _t, dev, host, rounded, within

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_chunkwise_gb300 import build
    build.build()
    ldn.load()


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    import torch
    yield
    assert ldn.ldn_get_device_status(torch.cuda.current_stream().cuda_stream) == ldn.LDN_OK


# ---- norms around a block ----
def gated_inputs(B, T, D, dtype, res, gate, gtype, seed=0):
    r = np.random.default_rng(seed)
    shape = {"none": None, "channel": (D,), "sequence": (B, 1, D), "token": (B, T, D)}[gate]
    return dict(x=rounded(r.normal(size=(B, T, D)), dtype), r=rounded(2 * r.normal(size=(B, T, D)), res),
                w=rounded(1 + 0.1 * r.normal(size=D), "f32"), wp=rounded(1 + 0.1 * r.normal(size=D), "f32"),
                gate=None if shape is None else rounded(r.normal(size=shape), gtype),
                dy=rounded(r.normal(size=(B, T, D)), dtype), dsum=rounded(r.normal(size=(B, T, D)), res))


GATED = [  # B, T, D, dtype, residual, gate, gate's type, sigmoid, post, pre, scale, dsum
    (1, 1, 1, "f32", "f32", "channel", "f32", False, True, True, 1.0, True),
    (1, 1, 64, "bf16", "bf16", "token", "bf16", True, True, True, 1.0, True),
    (2, 3, 7, "bf16", "f32", "sequence", "bf16", False, True, True, 0.5, True),
    (3, 5, 129, "f32", "f32", "none", "f32", False, True, True, 1.0, True),
    (2, 4, 1000, "bf16", "bf16", "channel", "f32", True, True, True, 2.0, False),
    (1, 70, 2048, "bf16", "f32", "token", "f32", False, True, True, 1.0, True),
    (5, 9, 2040, "bf16", "bf16", "sequence", "f32", True, True, True, 1.0, True),
    (1, 3, 4095, "f32", "f32", "sequence", "f32", True, True, True, -0.25, True),
    (2, 3, 4096, "bf16", "bf16", "channel", "f32", False, True, True, 1.0, True),
    (3, 1, 6001, "bf16", "f32", "channel", "bf16", False, True, True, 1.0, True),
    (1, 5, 8192, "bf16", "bf16", "token", "bf16", True, True, True, 1.0, True),
    (1, 4, 8192, "f32", "f32", "channel", "f32", False, True, True, 1.0, True),
    (2, 2, 9001, "bf16", "f32", "token", "bf16", False, True, True, 1.0, True),
    (1, 3, 16384, "f32", "f32", "sequence", "f32", False, True, True, 1.0, True),
    (1, 2, 16384, "bf16", "bf16", "channel", "f32", True, True, True, 1.0, False),
    (2, 30, 96, "bf16", "bf16", "channel", "f32", False, False, True, 1.0, True),
    (2, 30, 96, "bf16", "f32", "sequence", "bf16", True, True, False, 1.0, True),
    (2, 30, 96, "f32", "f32", "token", "f32", False, False, False, 0.5, True),
    (2, 30, 96, "bf16", "bf16", "none", "bf16", False, False, True, 1.0, False),
    (400, 3, 72, "bf16", "bf16", "sequence", "bf16", False, True, True, 1.0, True),
    (4, 300, 256, "f32", "f32", "sequence", "f32", True, True, True, 1.0, True),
    (1, 1500, 264, "bf16", "f32", "channel", "f32", False, True, True, 1.0, True)]


@pytest.mark.parametrize("case", GATED)
def test_gated_add_rmsnorm_and_backward(case):
    B, T, D, dtype, res, gate, gtype, sig, post, pre, scale, add = case
    p = gated_inputs(B, T, D, dtype, res, gate, gtype)
    w, wp, dsum = p["w"] if pre else None, p["wp"] if post else None, p["dsum"] if add else None
    t = dict(x=dev(p["x"], dtype), w=dev(w), wp=dev(wp), gate=dev(p["gate"], gtype))
    y, s = ldn.gated_add_rmsnorm(t["x"], dev(p["r"], res), t["w"], t["wp"], t["gate"], residual_scale=scale,
                                 gate_sigmoid=sig, eps=EPS)
    assert s.dtype == _t(res) and (y is None) == (not pre)
    dy = p["dy"] if pre else None
    if dy is None and dsum is None:
        dsum = p["dsum"]
    g = ldn.gated_add_rmsnorm_backward(dev(dy, dtype), t["x"], s, t["w"], t["wp"], t["gate"], dev(dsum, res),
                                       residual_scale=scale, gate_sigmoid=sig, eps=EPS)
    hs = host(s)
    own, want = ref.gated(p["x"], p["r"], w, wp, p["gate"], scale, sig, EPS, hs)
    b = ref.gated_bounds(p["x"], p["r"], w, wp, p["gate"], scale, sig, EPS, hs, dtype, res, gtype, dy, dsum)
    within(s, own, b["s"], "s")
    if pre:
        assert y.dtype == _t(dtype)
        within(y, want, b["y"], "y")
    for k, v in ref.gated_bwd(dy, p["x"], hs, w, wp, p["gate"], dsum, scale, sig, EPS).items():
        within(g[k], v, b[k], k)
    assert (g["dgate"] is None) == (gate == "none") and (g["dweight"] is None) == (not pre)
    assert (g["dpost_weight"] is None) == (not post)


def test_gated_add_rmsnorm_is_add_rmsnorm_without_a_gate():
    """s = x + r and its norm: the plain norm's sums, and its results up to the last step of the root."""
    import torch
    p = gated_inputs(1, 9, 520, "bf16", "bf16", "none", "bf16")
    x, r, w = dev(p["x"], "bf16"), dev(p["r"], "bf16"), dev(p["w"])
    y, s = ldn.gated_add_rmsnorm(x, r, w)
    y0, s0 = ldn.add_rmsnorm(x, r, w)
    assert torch.equal(s, s0) and torch.allclose(y.float(), y0.float(), rtol=2.0 ** -7, atol=0)


def test_gated_add_rmsnorm_in_place_unaligned_and_empty():
    import torch
    p = gated_inputs(2, 5, 65, "bf16", "bf16", "token", "bf16")
    args = lambda off: [dev(p[k], d, off=off) for k, d in (("x", "bf16"), ("r", "bf16"), ("w", "f32"),  # noqa: E731
                                                           ("wp", "f32"), ("gate", "bf16"))]
    want = ldn.gated_add_rmsnorm(*args(0), gate_sigmoid=True)
    for off in (1, 3):
        x, r, w, wp, gate = args(off)
        y, s = ldn.gated_add_rmsnorm(x, r, w, wp, gate, gate_sigmoid=True, residual_out=r)
        assert s is r and torch.equal(s, want[1]) and torch.equal(y, want[0])
    for shape, gshape in (((0, 64), (64,)), ((3, 0, 64), (3, 1, 64)), ((0, 64), (0, 64))):
        x = torch.zeros(shape, device="cuda")
        w, gate = torch.ones(64, device="cuda"), torch.ones(gshape, device="cuda")
        y, s = ldn.gated_add_rmsnorm(x, x, w, w, gate)
        assert y.shape == s.shape == shape
        g = ldn.gated_add_rmsnorm_backward(x, x, s, w, w, gate, gate_sigmoid=True)
        assert g["dx"].shape == shape and g["dgate"].shape == gshape
        assert not g["dgate"].any() and not g["dweight"].any() and not g["dpost_weight"].any()


def test_gated_add_rmsnorm_what_is_not_finite_stays_in_its_row():
    import torch
    for bad in (float("nan"), float("inf")):
        for D in (64, 300):
            p = gated_inputs(1, 6, D, "f32", "f32", "channel", "f32")
            x, r, w, wp, gate = (dev(p[k]) for k in ("x", "r", "w", "wp", "gate"))
            y0, s0 = ldn.gated_add_rmsnorm(x, r, w, wp, gate)
            x[0, 2, 5] = bad
            r[0, 4, 1] = bad
            y, s = ldn.gated_add_rmsnorm(x, r, w, wp, gate)
            keep = [0, 1, 3, 5]
            assert torch.equal(y[:, keep], y0[:, keep]) and torch.equal(s[:, keep], s0[:, keep])
            assert not torch.isfinite(s[0, 2, 5]) and not torch.isfinite(s[0, 4, 1])
            assert not torch.isfinite(y[0, [2, 4]]).all(-1).any()


# ---- projections ----
def linear_inputs(M, K, N, dtype, out, bias, seed=0):
    r = np.random.default_rng(seed)
    return dict(x=rounded(r.normal(size=(M, K)), dtype), w=rounded(r.normal(size=(N, K)) * K ** -0.5, dtype),
                b=rounded(0.5 * r.normal(size=N), dtype) if bias else None, r=rounded(r.normal(size=(M, N)), out),
                dy=rounded(r.normal(size=(M, N)), out))


SIZES = [(1, 1, 1), (1, 8, 128), (1, 4096, 300), (3, 64, 129), (16, 520, 1000), (17, 100, 77), (33, 63, 256), (64, 2048, 64),
         (65, 72, 136), (130, 1000, 333), (128, 256, 512), (257, 129, 255), (300, 65, 1), (1000, 16, 48), (513, 640, 1100)]
KINDS = [("bf16", None, None, True), ("bf16", "bf16", "silu", False), ("bf16", "f32", "gelu", True),
         ("bf16", "f32", None, False), ("f32", None, "gelu", True), ("f32", "f32", None, False), ("f32", "f32", "silu", True)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("dtype,res,act,bias", KINDS)
def test_linear_and_backward(M, K, N, dtype, res, act, bias):
    out = res or dtype
    p = linear_inputs(M, K, N, dtype, out, bias)
    r = p["r"] if res else None
    x, w = dev(p["x"], dtype), dev(p["w"], dtype)
    y, z = ldn.linear(x, w, dev(p["b"], dtype), dev(r, out) if res else None, activation=act, save_z=True)
    assert y.dtype == _t(out) and z.dtype == _t(dtype)
    b = ref.linear_bounds(p["x"], p["w"], p["b"], r, act, dtype, out, p["dy"])
    wy, wz = ref.linear(p["x"], p["w"], p["b"], r, act)
    within(y, wy, b["y"], "y")
    within(z, wz, b["z"], "z")
    g = ldn.linear_backward(dev(p["dy"], out), x, w, z if act else None, activation=act, bias=True)
    want, _ = ref.linear_bwd(p["dy"], p["x"], p["w"], wz, act)
    for k, v in want.items():
        assert g[k].dtype == _t(dtype)
        within(g[k], v, b[k], k)


@pytest.mark.parametrize("M,K,N", [(5, 20000, 130), (300, 8200, 40)])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
def test_linear_long_sums(M, K, N, dtype, out):
    """Over many chunks of k.  Where sums are kept the norm of the difference is within 64 steps of 2^-23 of
    the result's: a chunk of 1024 products has 64 additions in tensor memory, each cut off by a step of its
    partial sum at most."""
    import torch
    p = linear_inputs(M, K, N, dtype, out, False)
    r = dev(p["r"], out)
    y = ldn.linear(dev(p["x"], dtype), dev(p["w"], dtype), None, r)
    b = ref.linear_bounds(p["x"], p["w"], None, p["r"], None, dtype, out)
    want = ref.linear(p["x"], p["w"], None, p["r"], None)[0]
    within(y, want, b["y"], "y")
    if out == "f32":
        assert np.linalg.norm(host(y) - want) <= 64 * 2.0 ** -23 * np.linalg.norm(want)
    assert torch.equal(y, ldn.linear(dev(p["x"], dtype), dev(p["w"], dtype), None, r))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_strides_addresses_and_shapes(dtype):
    """Slices of wider rows, odd addresses, leading dimensions: the values of contiguous ones, bit for
    bit, and nothing outside the slices read (NaN there)."""
    import torch
    p = linear_inputs(12, 72, 50, dtype, dtype, True)
    x, w, b = dev(p["x"], dtype), dev(p["w"], dtype), dev(p["b"], dtype)
    want = ldn.linear(x, w, b, activation="silu")
    dy = dev(p["dy"], dtype)
    _, z = ldn.linear(x, w, b, activation="silu", save_z=True)
    gwant = ldn.linear_backward(dy, x, w, z, activation="silu", bias=True)
    for pad, off in ((8, 0), (8, 8), (3, 1), (0, 1), (5, 0)):
        x2, w2 = dev(p["x"], dtype, pad=pad, off=off), dev(p["w"], dtype, pad=pad, off=off)
        assert torch.equal(ldn.linear(x2, w2, b, activation="silu"), want), (pad, off)
        g = ldn.linear_backward(dev(p["dy"], dtype, off=off), x2, w2, z, activation="silu", bias=True)
        for k in gwant:
            assert torch.equal(g[k], gwant[k]), (pad, off, k)
    assert torch.equal(ldn.linear(x.view(3, 4, 72), w, b, activation="silu"), want.view(3, 4, 50))
    one = ldn.linear(x[5], w, b, activation="silu")
    assert one.shape == (50,) and torch.allclose(one.float(), want[5].float(), rtol=2.0 ** -7, atol=1e-5)
    out = torch.empty_like(want)
    assert ldn.linear(x, w, b, activation="silu", out=out) is out and torch.equal(out, want)


def test_linear_into_the_residual_and_no_rows():
    import torch
    p = linear_inputs(40, 64, 72, "bf16", "f32", True)
    x, w, b, r = dev(p["x"], "bf16"), dev(p["w"], "bf16"), dev(p["b"], "bf16"), dev(p["r"])
    want = ldn.linear(x, w, b, r, activation="gelu")
    assert ldn.linear(x, w, b, r, activation="gelu", out=r) is r and torch.equal(r, want)
    for dtype in (torch.bfloat16, torch.float32):
        x, w = torch.zeros(0, 64, device="cuda", dtype=dtype), torch.ones(72, 64, device="cuda", dtype=dtype)
        assert ldn.linear(x, w).shape == (0, 72)
        g = ldn.linear_backward(torch.zeros(0, 72, device="cuda", dtype=dtype), x, w, bias=True)
        assert g["dx"].shape == (0, 64) and not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.parametrize("M", [4, 300])
def test_linear_what_is_not_finite(M):
    """fp32 through planes of bf16 as in fp32: an infinity is one, of its sign, but against a zero; a
    NaN stays in its row and column; the largest numbers do not overflow."""
    import torch
    p = linear_inputs(M, 130, 70, "f32", "f32", False)
    x, w = dev(p["x"]), dev(p["w"])
    want = ldn.linear(x, w)
    x[1, 3] = float("inf")
    x[2, 7] = float("nan")
    w[5, 3] = 0.0
    w[6, 9] = float("-inf")
    y = ldn.linear(x, w)
    rows = [i for i in range(M) if i not in (1, 2)]
    cols = [j for j in range(70) if j not in (5, 6)]
    assert torch.equal(y[rows][:, cols], want[rows][:, cols])
    assert torch.isnan(y[2]).all() and torch.isnan(y[1, 5])
    assert torch.equal(y[1, cols], torch.copysign(torch.full_like(y[1, cols], float("inf")), w[cols, 3]))
    assert torch.equal(y[rows, 6], torch.copysign(torch.full_like(y[rows, 6], float("inf")), -x[rows, 9]))
    big = torch.zeros(2, 8, device="cuda")
    big[0, 0], big[1, 1] = torch.finfo(torch.float32).max, torch.finfo(torch.float32).min
    eye = torch.eye(8, device="cuda")
    assert torch.equal(ldn.linear(big, eye), big)


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 64, 256), (7, 100, 33), (16, 512, 640), (64, 4096, 200), (130, 272, 129),
                                   (300, 1000, 520)])
@pytest.mark.parametrize("res,act,bias", [(None, None, True), ("bf16", "silu", False), ("f32", "gelu", True)])
def test_linear_e4m3(M, K, N, res, act, bias):
    import torch
    r = np.random.default_rng(6)
    q = dev(rounded(r.normal(size=(M, K)) * 100, "f32")).clamp(-448, 448).to(torch.float8_e4m3fn)
    wq = dev(rounded(r.normal(size=(N, K)) * 100, "f32")).clamp(-448, 448).to(torch.float8_e4m3fn)
    sx, sw = rounded(np.exp(r.normal(size=M)) / 100, "f32"), rounded(np.exp(r.normal(size=N)) / 100, "f32")
    b, re = rounded(r.normal(size=N), "bf16") if bias else None, rounded(r.normal(size=(M, N)), res or "bf16")
    y = ldn.linear_e4m3(q, dev(sx), wq, dev(sw), dev(b, "bf16"), dev(re, res) if res else None, activation=act)
    assert y.dtype == _t(res or "bf16")
    x, w = host(q.float()) * sx[:, None], host(wq.float()) * sw[:, None]
    want, z = ref.linear(x, w, b, re if res else None, act)
    bound = ref.linear_bounds(x, w, b, re if res else None, act, "bf16", res or "bf16")["y"]
    # the scales' products: three roundings more, before the bias
    within(y, want, bound + ref.SLOPE * 4 * ref.U * np.abs(z - (0 if b is None else b)), "y")


def test_linear_e4m3_of_slices():
    import torch
    r = np.random.default_rng(7)
    q = torch.from_numpy(r.normal(size=(20, 80)) * 50).to("cuda").to(torch.float8_e4m3fn)
    w = torch.from_numpy(r.normal(size=(30, 80)) * 50).to("cuda").to(torch.float8_e4m3fn)
    sx, sw = torch.rand(20, device="cuda"), torch.rand(30, device="cuda")
    for a, b in ((0, 64), (16, 80), (3, 70), (1, 80)):
        want = ldn.linear_e4m3(q[:, a:b].contiguous(), sx, w[:, a:b].contiguous(), sw)
        assert torch.equal(ldn.linear_e4m3(q[:, a:b], sx, w[:, a:b], sw), want), (a, b)


# ---- streams and graphs ----
def a_block(p, t, ws):
    """One block's steps as a model takes them: the norm in 8 bits, the projection into the mixer, the
    projection out of it onto the stream, and the way to the next block."""
    q, sc, s = ldn.add_rmsnorm_e4m3(t["x"], t["r"], ws["norm"])
    u = ldn.linear_e4m3(q, sc, ws["in8"], ws["in_scale"], activation="silu")
    o = ldn.linear(u, ws["out"], ws["bias"])
    y, s2 = ldn.gated_add_rmsnorm(o, s, ws["norm2"], ws["post"], ws["gate"], residual_scale=0.5)
    return y, s2


def block_inputs(rows, seed=0):
    import torch
    r = np.random.default_rng(seed)
    D, H = 256, 640
    f = lambda *s, k=1.0: torch.from_numpy(r.normal(size=s) * k).float().cuda()  # noqa: E731
    w = f(H, D, k=D ** -0.5)
    scale = w.abs().amax(1) / 448
    ws = dict(norm=1 + f(D, k=0.1), in8=(w / scale[:, None]).to(torch.float8_e4m3fn), in_scale=scale,
              out=f(D, H, k=H ** -0.5).bfloat16(), bias=f(D, k=0.1).bfloat16(), norm2=1 + f(D, k=0.1),
              post=1 + f(D, k=0.1), gate=f(D))
    return dict(x=f(rows, D).bfloat16(), r=f(rows, D).bfloat16()), ws


@pytest.mark.parametrize("rows", [1, 5, 64, 700])
def test_a_block_with_its_projections(rows):
    """Against the same steps in 64 bits, each from what the step before stored."""
    t, ws = block_inputs(rows)
    q, sc, s = ldn.add_rmsnorm_e4m3(t["x"], t["r"], ws["norm"])
    u = ldn.linear_e4m3(q, sc, ws["in8"], ws["in_scale"], activation="silu")
    o = ldn.linear(u, ws["out"], ws["bias"])
    y, s2 = ldn.gated_add_rmsnorm(o, s, ws["norm2"], ws["post"], ws["gate"], residual_scale=0.5)
    x8 = host(q.float()) * host(sc)[:, None]
    w8 = host(ws["in8"].float()) * host(ws["in_scale"])[:, None]
    b = ref.linear_bounds(x8, w8, None, None, "silu", "bf16", "bf16")["y"]
    want, z = ref.linear(x8, w8, None, None, "silu")
    within(u, want, b + ref.SLOPE * 4 * ref.U * np.abs(z), "u")
    hw = [host(ws[k]) for k in ("out", "bias", "norm2", "post", "gate")]
    within(o, ref.linear(host(u), hw[0], hw[1], None, None)[0],
           ref.linear_bounds(host(u), hw[0], hw[1], None, None, "bf16", "bf16")["y"], "o")
    b = ref.gated_bounds(host(o), host(s), hw[2], hw[3], hw[4], 0.5, False, 1e-6, host(s2), "bf16", "bf16")
    own, wy = ref.gated(host(o), host(s), hw[2], hw[3], hw[4], 0.5, False, 1e-6, host(s2))
    within(s2, own, b["s"], "s2")
    within(y, wy, b["y"], "y")


def test_calls_on_another_stream_and_side_by_side():
    import torch
    sets = [block_inputs(n, seed=n) for n in (3, 64, 300)]
    want = [a_block(None, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for st, s in zip(streams, sets):
        with torch.cuda.stream(st):
            got.append(a_block(None, *s))
    x, w = sets[0][0]["x"].float(), sets[0][1]["out"].float().t().contiguous()
    alone = ldn.linear(x, w)
    torch.cuda.synchronize()
    over = ldn.linear(x, w, stream=streams[1])      # with a workspace of that stream's
    torch.cuda.synchronize()
    assert torch.equal(alone, over)
    for a, b in zip(got, want):
        assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_calls_captured_and_replayed():
    """Two graphs of the same calls, replayed in turn and on inputs that change between."""
    import torch
    t, ws = block_inputs(70)
    f32 = [torch.randn(70, 256, device="cuda"), torch.randn(100, 256, device="cuda")]
    dy = torch.randn(70, 100, device="cuda")

    def all_of_it():
        y, s = a_block(None, t, ws)
        z = ldn.linear(*f32, activation="gelu", save_z=True)
        g = ldn.linear_backward(dy, *f32, z[1], activation="gelu", bias=True)
        n = ldn.gated_add_rmsnorm_backward(y, t["x"], s, ws["norm2"], ws["post"], ws["gate"], s)
        return [y, s, *z, *g.values(), *n.values()]
    all_of_it()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = all_of_it()
        graphs.append((g, out))
    for seed in range(3):
        t["x"].copy_(block_inputs(70, seed=seed + 10)[0]["x"])
        f32[0].normal_()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = all_of_it()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---- refusals of the torch layer ----
def test_torch_layer_refuses():
    import torch
    d = "cuda"
    x, w, b = torch.zeros(4, 64, device=d), torch.zeros(32, 64, device=d), torch.zeros(32, device=d)
    bf = lambda t: t.bfloat16()  # noqa: E731
    for bad, err in (((x.cpu(), w), TypeError), ((x, w.cpu()), TypeError), ((x, bf(w)), TypeError),
                     ((x.half(), w.half()), TypeError), ((x, w[:, :63]), ValueError), ((x, w[0]), ValueError),
                     ((x, w, b[:31]), ValueError), ((x, w, bf(b)), TypeError), ((x, w, b, x), ValueError),
                     ((x, w, b, torch.zeros(4, 32, device=d).half()), TypeError), ((x, None), TypeError),
                     ((x.t(), w), ValueError), ((x[:, ::2], w[:, ::2]), ValueError), ((torch.tensor(1.0, device=d), w), ValueError),
                     ((x, w, b, torch.zeros(32, 4, device=d).t()), ValueError),
                     ((x[:, :0], w[:, :0]), ldn.LdnError), ((x, w[:0]), ldn.LdnError),
                     ((x, w, None, bf(torch.zeros(4, 32, device=d))), ldn.LdnError)):
        with pytest.raises(err):
            ldn.linear(*bad)
    with pytest.raises(ValueError):
        ldn.linear(x, w, activation="relu")
    with pytest.raises(ValueError):
        ldn.linear(x, w, out=torch.zeros(4, 33, device=d))
    with pytest.raises(ldn.LdnError):
        ldn.linear(x[:, :32], w[:, :32], out=x.view(-1)[:128].view(4, 32))
    with pytest.raises(ValueError):
        ldn.linear(x, w, stream="main")
    dy = torch.zeros(4, 32, device=d)
    for bad, kw, err in (((dy, x, w), dict(activation="silu"), TypeError), ((dy.t(), x, w), {}, ValueError),
                         ((dy, x, w, bf(dy)), dict(activation="silu"), TypeError), ((bf(dy), x, w), {}, ldn.LdnError),
                         ((dy[:3], x, w), {}, ValueError)):
        with pytest.raises(err):
            ldn.linear_backward(*bad, **kw)
    q, wq, s = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), torch.ones(4, device=d)
    for bad, err in (((x, s, wq, b), TypeError), ((q, s, w, b), TypeError), ((q, s[:3], wq, b), ValueError),
                     ((q, s, wq, b[:3]), ValueError), ((q, None, wq, b), TypeError), ((q, s, wq, b, b), TypeError)):
        with pytest.raises(err):
            ldn.linear_e4m3(*bad)
    n = torch.ones(64, device=d)
    for bad, err in (((x, x[:3], n), ValueError), ((x, None, n), TypeError), ((x, x, n[:3]), ValueError),
                     ((x, x, n, n, torch.ones(2, 64, device=d)), ValueError), ((x, x, n, n, torch.ones(4, 1, device=d)), ValueError),
                     ((x, bf(x), n), ldn.LdnError), ((x, x, n, n, bf(n)), ldn.LdnError), ((x.t(), x.t(), n[:4]), ValueError),
                     ((x, x, n, n, torch.ones(1, 4, 64, device=d)), ValueError)):
        with pytest.raises(err):
            ldn.gated_add_rmsnorm(*bad)
    with pytest.raises(ValueError):
        ldn.gated_add_rmsnorm(x, x, None, n, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        ldn.gated_add_rmsnorm_backward(None, x, x, n)
    with pytest.raises(ValueError):
        ldn.gated_add_rmsnorm_backward(x, x, x, None)
    with pytest.raises(ldn.LdnError):
        ldn.gated_add_rmsnorm(x, x, n, residual_scale=float("inf"))


def test_calls_that_record_no_gradient_warn():
    import torch
    x, w = torch.zeros(4, 64, device="cuda", requires_grad=True), torch.ones(64, device="cuda")
    with pytest.warns(UserWarning, match="autograd.linear"):
        ldn.linear(x, torch.zeros(8, 64, device="cuda"))
    with pytest.warns(UserWarning, match="autograd.gated_add_rmsnorm"):
        ldn.gated_add_rmsnorm(x, x.detach(), w)


# ---- autograd ----
def leaf(t):
    return None if t is None else t.detach().clone().requires_grad_()


@pytest.mark.parametrize("gate,pre", [("none", True), ("channel", True), ("sequence", False), ("token", True)])
def test_autograd_gated_add_rmsnorm(gate, pre):
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    p = gated_inputs(2, 6, 72, "bf16", "f32", gate, "f32")
    a = [leaf(dev(p[k], d)) for k, d in (("x", "bf16"), ("r", "f32"), ("w", "f32"), ("wp", "f32"), ("gate", "f32"))]
    if not pre:
        a[2] = None
    y, s = ag.gated_add_rmsnorm(*a, residual_scale=0.5, gate_sigmoid=True)
    ds = torch.randn_like(s)
    dy = torch.randn_like(y) if pre else None
    torch.autograd.backward([y, s] if pre else [s], [dy, ds] if pre else [ds])
    d = [None if t is None else t.detach() for t in a]
    g = ldn.gated_add_rmsnorm_backward(dy, d[0], s.detach(), d[2], d[3], d[4], ds, residual_scale=0.5, gate_sigmoid=True)
    for t, k in zip(a, ("dx", "dresidual", "dweight", "dpost_weight", "dgate")):
        assert (t is None) == (g[k] is None) and (t is None or torch.equal(t.grad, g[k])), k
    if pre:     # the sum alone, and y alone
        for use in (0, 1):
            b = [leaf(t) for t in a]
            out = ag.gated_add_rmsnorm(*b, residual_scale=0.5, gate_sigmoid=True)
            out[use].backward((dy, ds)[use])
            want = ldn.gated_add_rmsnorm_backward((dy, torch.zeros_like(dy))[use], d[0], s.detach(), d[2], d[3], d[4],
                                                  (None, ds)[use], residual_scale=0.5, gate_sigmoid=True)
            assert torch.equal(b[0].grad, want["dx"]) and torch.equal(b[1].grad, want["dresidual"])


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_autograd_linear(act):
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    p = linear_inputs(30, 64, 40, "bf16", "f32", True)
    a = [leaf(dev(p[k], d)) for k, d in (("x", "bf16"), ("w", "bf16"), ("b", "bf16"), ("r", "f32"))]
    y = ag.linear(*a, activation=act)
    dy = dev(p["dy"])
    y.backward(dy)
    d = [t.detach() for t in a]
    z = ldn.linear(*d, activation=act, save_z=True)[1] if act else None
    g = ldn.linear_backward(dy, d[0], d[1], z, activation=act, bias=True)
    for t, k in zip(a, ("dx", "dweight", "dbias")):
        assert torch.equal(t.grad, g[k]), k
    assert torch.equal(a[3].grad, dy)
    x = leaf(a[0])      # one gradient alone
    ag.linear(x, d[1], activation=act).float().sum().backward()
    assert x.grad is not None
    with pytest.raises(RuntimeError):
        x = leaf(a[0])
        (gx,) = torch.autograd.grad(ag.linear(x, leaf(d[1]), activation=act).float().square().sum(), x, create_graph=True)
        gx.float().sum().backward()


def test_autograd_of_a_chain_against_differentiation_in_64_bits():
    """norm -> projection -> gelu -> projection -> gate and norms, in fp32, against torch's own
    differentiation of the formulas in 64 bits."""
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    torch.manual_seed(0)
    D, H, M = 72, 130, 50
    f = lambda *s, k=1.0: torch.randn(*s, device="cuda") * k  # noqa: E731
    names = dict(x=f(M, D), r=f(M, D), n1=1 + f(D, k=0.1), w1=f(H, D, k=D ** -0.5), b1=f(H, k=0.1), w2=f(D, H, k=H ** -0.5),
                 n2=1 + f(D, k=0.1), n3=1 + f(D, k=0.1), gate=f(D))
    dy, ds = f(M, D), f(M, D)

    def own(p):
        y, s = ag.add_rmsnorm(p["x"], p["r"], p["n1"])
        o = ag.linear(ag.linear(y, p["w1"], p["b1"], activation="gelu"), p["w2"])
        return ag.gated_add_rmsnorm(o, s, p["n3"], p["n2"], p["gate"], residual_scale=0.5, gate_sigmoid=True)

    def plain(p):
        norm = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
        s = p["x"] + p["r"]
        o = torch.nn.functional.gelu(norm(s, p["n1"]) @ p["w1"].t() + p["b1"]) @ p["w2"].t()
        s2 = 0.5 * s + torch.sigmoid(p["gate"]) * norm(o, p["n2"])
        return norm(s2, p["n3"]), s2
    a = {k: leaf(v) for k, v in names.items()}
    b = {k: leaf(v.double()) for k, v in names.items()}
    for out, p in ((own(a), a), (plain(b), b)):
        torch.autograd.backward(list(out), [dy.to(out[0].dtype), ds.to(out[0].dtype)])
    # fp32 through five steps: sums of at most 130 products, each step a few dozen roundings at 2^-24
    for k in names:
        rel = (a[k].grad.double() - b[k].grad).norm() / b[k].grad.norm()
        assert rel < 300 * 2.0 ** -24, (k, rel.item())
