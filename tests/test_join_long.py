"""The operators that join blocks at sizes where a block walks many rows or tiles: rows through the ring
in shared memory, tiles of pairs of blocks, split tiles, results staged in shared memory and not, against
the 64-bit definitions with the bounds of tests/_join_ref.py."""
import os
import subprocess

import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from tests import _join_ref as ref
from tests.test_join_parity import EPS, gated_inputs, linear_inputs
from tests.test_mixer_parity import _t, dev, host, within

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_chunkwise_gb300 import build
    build.build()
    ldn.load()


# ---- norms: B, T, D, dtype, residual, gate, gate's type, sigmoid, post, pre, scale, dsum ----
GATED = [
    (1, 1400, 2048, "bf16", "f32", "token", "bf16", True, True, True, 1.0, True),
    (1, 700, 4096, "bf16", "bf16", "channel", "f32", False, True, True, 0.5, True),
    (2, 650, 4096, "f32", "f32", "token", "f32", False, True, True, 1.0, True),
    (3, 460, 2040, "bf16", "bf16", "sequence", "f32", True, True, True, 1.0, False),
    (900, 3, 1024, "bf16", "f32", "sequence", "bf16", False, True, True, 1.0, True),
    (7, 391, 1024, "f32", "f32", "sequence", "f32", False, False, True, 2.0, True),
    (1, 2500, 1032, "bf16", "bf16", "none", "bf16", False, True, False, 1.0, True),
    (1, 400, 8192, "bf16", "f32", "channel", "bf16", True, True, True, 1.0, True),
    (2, 310, 8192, "f32", "f32", "token", "f32", False, False, False, 1.0, True),
    (1, 1300, 1025, "bf16", "f32", "channel", "f32", False, True, True, 1.0, True)]


@gpu
@pytest.mark.parametrize("case", GATED)
def test_gated_add_rmsnorm_of_many_rows(case):
    import torch
    B, T, D, dtype, res, gate, gtype, sig, post, pre, scale, add = case
    p = gated_inputs(B, T, D, dtype, res, gate, gtype, seed=3)
    w, wp, dsum = p["w"] if pre else None, p["wp"] if post else None, p["dsum"] if add else None
    dy = p["dy"] if pre else None
    t = dict(x=dev(p["x"], dtype), w=dev(w), wp=dev(wp), gate=dev(p["gate"], gtype))
    kw = dict(residual_scale=scale, gate_sigmoid=sig, eps=EPS)
    y, s = ldn.gated_add_rmsnorm(t["x"], dev(p["r"], res), t["w"], t["wp"], t["gate"], **kw)
    args = dev(dy, dtype), t["x"], s, t["w"], t["wp"], t["gate"], dev(dsum, res)
    g = ldn.gated_add_rmsnorm_backward(*args, **kw)
    hs = host(s)
    own, want = ref.gated(p["x"], p["r"], w, wp, p["gate"], scale, sig, EPS, hs)
    b = ref.gated_bounds(p["x"], p["r"], w, wp, p["gate"], scale, sig, EPS, hs, dtype, res, gtype, dy, dsum)
    within(s, own, b["s"], "s")
    if pre:
        within(y, want, b["y"], "y")
    for k, v in ref.gated_bwd(dy, p["x"], hs, w, wp, p["gate"], dsum, scale, sig, EPS).items():
        within(g[k], v, b[k], k)
    again = ldn.gated_add_rmsnorm_backward(*args, **kw)
    for k, v in g.items():
        assert v is None or torch.equal(v, again[k]), k
    assert ldn.ldn_get_device_status(torch.cuda.current_stream().cuda_stream) == ldn.LDN_OK


# ---- projections: M, K, N, dtype, residual, activation, bias, z ----
LINEAR = [
    (2049, 520, 1032, "bf16", None, None, True, False),
    (2049, 520, 1032, "bf16", None, "gelu", True, True),
    (2049, 520, 1032, "bf16", "bf16", "silu", False, False),
    (2049, 520, 1032, "bf16", "bf16", "silu", True, True),
    (2049, 520, 1032, "bf16", "f32", "gelu", True, False),
    (2049, 520, 1032, "bf16", "f32", "gelu", True, True),
    (2100, 2056, 1028, "bf16", "f32", None, False, False),
    (2100, 1100, 1004, "f32", "f32", "silu", True, False),
    (2100, 300, 1004, "f32", None, "gelu", True, True),
    (2111, 136, 2051, "bf16", "bf16", "gelu", True, False),
    (5000, 64, 2056, "bf16", "bf16", None, True, False),
    (20000, 72, 200, "bf16", None, None, False, False),
    (40, 4096, 4096, "bf16", "bf16", None, True, False),
    (100, 2048, 2048, "bf16", "f32", "silu", True, True),
    (20, 2048, 512, "f32", "f32", None, True, False)]


@gpu
@pytest.mark.parametrize("case", LINEAR)
def test_linear_and_backward_of_many_tiles(case):
    import torch
    M, K, N, dtype, res, act, bias, save = case
    out = res or dtype
    p = linear_inputs(M, K, N, dtype, out, bias, seed=4)
    r = p["r"] if res else None
    x, w = dev(p["x"], dtype), dev(p["w"], dtype)
    y = ldn.linear(x, w, dev(p["b"], dtype), dev(r, out) if res else None, activation=act, save_z=save)
    y, z = y if save else (y, None)
    b = ref.linear_bounds(p["x"], p["w"], p["b"], r, act, dtype, out, p["dy"])
    wy, wz = ref.linear(p["x"], p["w"], p["b"], r, act)
    within(y, wy, b["y"], "y")
    if save:
        within(z, wz, b["z"], "z")
    if res:     # in place: a tile's residual is read before the tile is written, and no other's is
        same = dev(r, out)
        ldn.linear(x, w, dev(p["b"], dtype), same, activation=act, out=same)
        assert torch.equal(same, y)
    if act is None or save:
        args = dev(p["dy"], out), x, w, z
        g = ldn.linear_backward(*args, activation=act, bias=True)
        want, _ = ref.linear_bwd(p["dy"], p["x"], p["w"], wz, act)
        for k, v in want.items():
            within(g[k], v, b[k], k)
        again = ldn.linear_backward(*args, activation=act, bias=True)
        assert all(torch.equal(g[k], again[k]) for k in g)
    assert ldn.ldn_get_device_status(torch.cuda.current_stream().cuda_stream) == ldn.LDN_OK


@gpu
@pytest.mark.parametrize("M,K,N,res,act", [(2049, 1040, 1032, "bf16", None), (2049, 1040, 1032, "f32", "gelu"),
                                           (2500, 272, 2051, None, "silu"), (33, 4096, 2048, "bf16", None)])
def test_linear_e4m3_of_many_tiles(M, K, N, res, act):
    import torch
    r = np.random.default_rng(8)
    q = dev(r.normal(size=(M, K)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    wq = dev(r.normal(size=(N, K)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    sx, sw = dev(np.exp(r.normal(size=M)) / 1e4), dev(np.exp(r.normal(size=N)) / 1e4)
    b, re = dev(r.normal(size=N), "bf16"), dev(r.normal(size=(M, N)), res or "bf16")
    y = ldn.linear_e4m3(q, sx, wq, sw, b, re if res else None, activation=act)
    x, w = host(q.float()) * host(sx)[:, None], host(wq.float()) * host(sw)[:, None]
    hb, hr = host(b), host(re) if res else None
    want, z = ref.linear(x, w, hb, hr, act)
    bound = ref.linear_bounds(x, w, hb, hr, act, "bf16", res or "bf16")["y"]
    within(y, want, bound + ref.SLOPE * 4 * ref.U * np.abs(z - hb), "y")


def test_the_cases_take_every_cut(tmp_path):
    """Pairs of blocks, single ones and split tiles are among the forward's cuts of the cases above."""
    from gated_delta_rule_chunkwise_gb300 import build as ldn_build
    src = tmp_path / "plan.cpp"
    src.write_text('#include <cstdio>\n#include "linear_plan.h"\nint main(){ long long i, j; int k, p, r;\n'
                   'while (scanf("%lld %lld %d %d %d", &i, &j, &k, &p, &r) == 5) {\n'
                   'ldn::linear::Plan q = ldn::linear::plan_for(i, j, k, p, false, r, 152);\n'
                   'printf("%d %d %d\\n", q.bn, q.split, q.pair); } }\n')
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ldn_build.CSRC), str(src), "-o", exe], check=True)
    rows = "\n".join(f"{N} {M} {-(-K // 64)} {6 if d == 'f32' else 1} {int((res or d) == 'f32')}"
                     for M, K, N, d, res, *_ in LINEAR)
    out = subprocess.run([exe], input=rows, capture_output=True, text=True, check=True).stdout.split()
    split, pair = set(map(int, out[1::3])), set(map(int, out[2::3]))
    assert pair == {0, 1} and 1 in split and len(split) > 1


@gpu
def test_pairs_and_splits_side_by_side():
    """Products of all kinds on several streams at once: what they give alone."""
    import torch
    sets = []
    for i, (M, K, N) in enumerate([(2048, 1024, 2048), (16, 4096, 2048), (300, 512, 512), (3000, 256, 1000)]):
        g = torch.Generator(device="cuda").manual_seed(i)
        sets.append([torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((M, K), (N, K), (M, N))])
    want = [(ldn.linear(x, w, None, r), ldn.linear_backward(r, x, w)) for x, w, r in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, (x, w, r) in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append((ldn.linear(x, w, None, r), ldn.linear_backward(r, x, w)))
        torch.cuda.synchronize()
        for (a, ga), (b, gb) in zip(got, want):
            assert torch.equal(a, b) and torch.equal(ga["dx"], gb["dx"]) and torch.equal(ga["dweight"], gb["dweight"])
    assert all(y.dtype == _t("bf16") for y, _ in want)


@gpu
def test_a_chain_of_calls_sees_what_each_wrote():
    """Blocks of a call start while the one before drains: each still reads what that one wrote, and writes
    nothing that it still reads.  Buffers are reused in turn, many times over."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    f = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    M, D, H = 256, 512, 1024
    w1, w2 = (f(H, D) * D ** -0.5).bfloat16(), (f(D, H) * H ** -0.5).bfloat16()
    n = 1 + 0.1 * f(D)
    x0 = f(M, D).bfloat16()

    def chain(sync):
        s, y = x0.clone(), x0.clone()
        u, o = torch.empty(M, H, device="cuda", dtype=torch.bfloat16), torch.empty_like(y)
        for _ in range(40):
            ldn.linear(y, w1, activation="silu", out=u)
            if sync:
                torch.cuda.synchronize()
            ldn.linear(u, w2, out=o)
            if sync:
                torch.cuda.synchronize()
            ldn.gated_add_rmsnorm(o, s, n, n, residual_scale=0.7, out=y, residual_out=s)
            if sync:
                torch.cuda.synchronize()
        return y, s
    a, b = chain(True), chain(False)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("shifted", ["y", "residual", "z", "all"])
def test_linear_results_at_any_address(out, shifted):
    """y, residual and z that start at odd elements: the same values bit for bit as at aligned ones, and
    nothing written around y."""
    import torch
    M, K, N = 2049, 264, 1032
    p = linear_inputs(M, K, N, "bf16", out, True, seed=9)
    x, w, b, r = (dev(p[k], d) for k, d in (("x", "bf16"), ("w", "bf16"), ("b", "bf16"), ("r", out)))
    want = ldn.linear(x, w, b, r, activation="silu")
    _, wz = ldn.linear(x, w, b, activation="silu", save_z=True)

    def at(t, move):
        flat = torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device="cuda")
        v = flat[move:move + t.numel()].view(t.shape)
        v.copy_(t)
        return v, flat
    y, flat = at(torch.zeros_like(want), int(shifted in ("y", "all")))
    r2, _ = at(r, int(shifted in ("residual", "all")))
    z, _ = at(torch.zeros_like(wz), int(shifted in ("z", "all")))
    st = ldn.ldn_linear(x.data_ptr(), K, w.data_ptr(), K, b.data_ptr(), r2.data_ptr(), y.data_ptr(), z.data_ptr(), M, K, N,
                        ldn.LDN_ACT_SILU, ldn.LDN_BF16, ldn.LDN_F32 if out == "f32" else ldn.LDN_BF16, None, 0,
                        torch.cuda.current_stream().cuda_stream)
    assert st == ldn.LDN_OK
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, wz)
    move = int(shifted in ("y", "all"))
    assert (flat[:move] == 7.0).all() and (flat[move + y.numel():] == 7.0).all()


@gpu
def test_autograd_linear_keeps_z_only_for_a_gradient():
    import torch
    from gated_delta_rule_chunkwise_gb300 import autograd as ag
    x, w = torch.randn(64, 256, device="cuda"), torch.randn(4096, 256, device="cuda")
    torch.cuda.synchronize()

    def grown(*a):
        base = torch.cuda.memory_allocated()
        y = ag.linear(*a, activation="gelu")
        return torch.cuda.memory_allocated() - base, y
    size = 64 * 4096 * 4
    assert grown(x, w)[0] == size and grown(x, w.requires_grad_())[0] == 2 * size
