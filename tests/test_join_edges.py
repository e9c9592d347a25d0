"""The operators that join blocks at the edges of what their documentation allows: outputs that are left out,
workspaces of exactly the stated size, the largest and smallest rows, very long sums."""
import itertools
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


# ---- the norms' gradient with outputs left out ----
def test_gated_workspace_holds_a_call_without_dgate():
    """Without dgate the rows are walked as without a gate: the stated size is no smaller than there."""
    f = ldn.ldn_gated_add_rmsnorm_backward_workspace_size
    cases = [(1530, 2048, 153), (7700, 4096, 77), (7700, 8192, 77), (5120, 4096, 80), (6400, 4096, 100),
             (1280, 2048, 160)]
    r = np.random.default_rng(0)
    for _ in range(3000):
        gates, each, D = (int(np.exp(r.uniform(0, np.log(n)))) for n in (2000, 300, 16384))
        cases.append((gates * each, int(r.choice([D, max(8, D // 8 * 8)])), gates))
    for rows, D, gates in cases:
        assert f(rows, D, gates) >= f(rows, D, 0), (rows, D, gates)


def c_backward(p, s, case, give, guard=1 << 20):
    """ldn_gated_add_rmsnorm_backward with the outputs `give` alone, on a workspace of exactly the stated size
    between guards; the other outputs are None."""
    import torch
    B, T, D, dtype, res, gate, gtype, sig, scale = case
    rows, gates = B * T, p["gate"].size // D
    t = dict(dy=dev(p["dy"], dtype), x=dev(p["x"], dtype), s=s, dsum=dev(p["dsum"], res), gate=dev(p["gate"], gtype),
             wp=dev(p["wp"]), w=dev(p["w"]))
    new = dict(dx=((B, T, D), dtype), dresidual=((B, T, D), res), dgate=(p["gate"].shape, gtype))
    out = {k: torch.empty(shape, dtype=_t(d), device="cuda") if k in give else None for k, (shape, d) in new.items()}
    out |= {k: torch.empty(D, device="cuda") for k in ("dpost_weight", "dweight")}
    need = ldn.ldn_gated_add_rmsnorm_backward_workspace_size(rows, D, gates)
    room = torch.full((guard + need + guard,), 0x5a, dtype=torch.uint8, device="cuda")
    q = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    codes = {"f32": ldn.LDN_F32, "bf16": ldn.LDN_BF16}
    st = ldn.ldn_gated_add_rmsnorm_backward(
        *(q(t[k]) for k in ("dy", "x", "s", "dsum", "gate", "wp", "w")),
        *(q(out[k]) for k in ("dx", "dresidual", "dgate", "dpost_weight", "dweight")), rows, D, gates, codes[gtype],
        int(sig), scale, codes[dtype], codes[res], EPS, room.data_ptr() + guard, need,
        torch.cuda.current_stream().cuda_stream)
    assert st == ldn.LDN_OK
    torch.cuda.synchronize()
    assert (room[:guard] == 0x5a).all() and (room[guard + need:] == 0x5a).all()
    return out


@gpu
@pytest.mark.parametrize("case", [  # B, T, D, dtype, residual, gate, gate's type, sigmoid, scale
    (153, 10, 2048, "bf16", "bf16", "sequence", "bf16", False, 1.0),
    (80, 11, 4096, "bf16", "f32", "sequence", "f32", True, 0.5),
    (77, 8, 8192, "f32", "f32", "sequence", "f32", False, 1.0),
    (160, 8, 333, "f32", "f32", "sequence", "f32", True, 1.0),
    (2, 300, 1024, "bf16", "f32", "channel", "f32", False, 1.0),
    (2, 400, 1024, "bf16", "bf16", "token", "bf16", True, 1.0)])
def test_gated_backward_with_outputs_left_out(case):
    """Each of dx, dresidual and dgate may be NULL: the others are what they are with all of them, and nothing
    is written around the workspace."""
    B, T, D, dtype, res, gate, gtype, sig, scale = case
    p = gated_inputs(B, T, D, dtype, res, gate, gtype, seed=5)
    _, s = ldn.gated_add_rmsnorm(dev(p["x"], dtype), dev(p["r"], res), dev(p["w"]), dev(p["wp"]), dev(p["gate"], gtype),
                                 residual_scale=scale, gate_sigmoid=sig, eps=EPS)
    hs = host(s)
    own = {k: p[k] for k in ("x", "r", "w", "wp", "gate")}
    b = ref.gated_bounds(*own.values(), scale, sig, EPS, hs, dtype, res, gtype, p["dy"], p["dsum"])
    want = ref.gated_bwd(p["dy"], p["x"], hs, p["w"], p["wp"], p["gate"], p["dsum"], scale, sig, EPS)
    names = ("dx", "dresidual", "dgate")
    for n in range(4):
        for give in itertools.combinations(names, n):
            for k, v in c_backward(p, s, case, give).items():
                if v is not None:
                    within(v, want[k], b[k], f"{k} of {give}")


@gpu
@pytest.mark.parametrize("size", [1e16, 1e-16])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,D", [(3, 64), (700, 1024), (2, 8192), (5, 777)])
def test_gated_gradient_of_large_and_small_rows(T, D, post, size):
    """One norm alone, without eps, of rows whose squares are in fp32's range but whose cubes are not: the
    gradient's second term, as large as the first over the root of D, is there."""
    p = gated_inputs(1, T, D, "f32", "f32", "none", "f32", seed=6)
    f = np.float32(size)
    x, r, dy = (np.float64(np.float32(p[k]) * f) for k in ("x", "r", "dy"))
    w, wp, dsum = (None, p["wp"], p["dsum"]) if post else (p["w"], None, None)
    dy = None if post else dy
    _, s = ldn.gated_add_rmsnorm(dev(x), dev(r), dev(w), dev(wp), eps=0.0)
    hs = host(s)
    g = ldn.gated_add_rmsnorm_backward(dev(dy), dev(x), s, dev(w), dev(wp), None, dev(dsum), eps=0.0)
    b = ref.gated_bounds(x, r, w, wp, None, 1.0, False, 0.0, hs, "f32", "f32", None, dy, dsum)
    want = ref.gated_bwd(dy, x, hs, w, wp, None, dsum, 1.0, False, 0.0)
    for k in ("dx", "dresidual", "dpost_weight" if post else "dweight"):
        within(g[k], want[k], b[k], k)


# ---- tensor memory ----
def test_accumulators_are_read_where_they_are_allocated(tmp_path):
    """Every load of the epilogue, 32 columns of promoted sums and 16 of others from where each half of a tile
    begins, lies inside its own accumulator of the two that the block allocates."""
    from gated_delta_rule_chunkwise_gb300 import build as ldn_build
    src = tmp_path / "columns.cpp"
    src.write_text('#include <cstdio>\n#include "linear_plan.h"\nint main(){ int bn, p;\n'
                   'while (scanf("%d %d", &bn, &p) == 2)\n'
                   'printf("%d %d\\n", ldn::linear::tensor_columns(bn, p), ldn::linear::half_columns(bn)); }\n')
    exe = str(tmp_path / "columns")
    subprocess.run(["g++", "-std=c++17", "-I", ldn_build.CSRC, str(src), "-o", exe], check=True)
    asked = [(bn, p) for bn in (16, 32, 64, 96, 128, 160, 192, 224, 256) for p in (0, 1)]
    out = subprocess.run([exe], input="\n".join(f"{b} {p}" for b, p in asked), capture_output=True, text=True,
                         check=True).stdout.split()
    for (bn, promote), cols, per in zip(asked, map(int, out[::2]), map(int, out[1::2])):
        assert cols in (32, 64, 128, 256, 512) and bn <= cols // 2 and per % 16 == 0 and per <= bn
        unit = 32 if promote else 16
        for first, n in ((0, min(per, bn)), (per, bn - per)):
            for c in range(0, n, unit):
                assert first + c + unit <= cols // 2, (bn, promote, first, c)


@gpu
@pytest.mark.parametrize("M", [1, 16, 17, 32, 33])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_tokens_over_many_chunks(M, dtype):
    """fp32 results of few tokens: narrow tiles whose sums are taken over both accumulators in turn, beside
    another product that fills the rest of the card."""
    import torch
    K, N = 8192, 520
    p = linear_inputs(M, K, N, dtype, "f32", True, seed=11)
    x, w, b, r = dev(p["x"], dtype), dev(p["w"], dtype), dev(p["b"], dtype), dev(p["r"])
    y = ldn.linear(x, w, b, r)
    bound = ref.linear_bounds(p["x"], p["w"], p["b"], p["r"], None, dtype, "f32")["y"]
    within(y, ref.linear(p["x"], p["w"], p["b"], p["r"], None)[0], bound, "y")
    wide = torch.randn(2048, 1024, device="cuda").bfloat16()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        ldn.linear(wide, wide, stream=other)
        assert torch.equal(ldn.linear(x, w, b, r), y)
    torch.cuda.synchronize()


# ---- bf16 results of very long sums ----
def tokens_of_one_sign(T, D, seed):
    """dy and x, whose rows are all the same, so that dweight is the columns' sums of dy times x's row."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    column = 1 + torch.rand(D, device="cuda", generator=g)
    x = (1 + torch.rand(D, device="cuda", generator=g)).bfloat16().repeat(T, 1)
    dy = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    for part in dy.split(1 << 16):
        part.copy_((0.5 + torch.rand(part.shape, device="cuda", generator=g)) * column)
    return dy, x


@gpu
def test_dweight_over_a_million_tokens():
    """What an addition in tensor memory cuts off is always towards zero: over sums of one sign it is the mean of
    the results' relative errors, in which their roundings to bf16 (at most 2^-8 each, of either sign, 2.4 million
    of them) leave 1e-5 at most.  A chunk of 65536 products is 4096 additions, and 32 more for those within one; in
    each the 16 products and the partial sum are cut off by a step of fp32 of the largest, 17 2^-23 of a partial
    sum that grows evenly: 4128 / 2 17 2^-23 of the chunk's at most, and as much of the whole sum."""
    import torch
    T, D = 1 << 20, 1536
    dy, x = tokens_of_one_sign(T, D, 12)
    got = ldn.linear_backward(dy, x, torch.zeros(D, D, dtype=torch.bfloat16, device="cuda"), dx=False)["dweight"]
    want = dy.sum(0, dtype=torch.float64)[:, None] * x[0].double()
    off = (got.double() - want) / want
    cut = 4128 / 2 * 17 * 2.0 ** -23
    assert off.abs().max().item() <= 2.0 ** -8 + cut
    assert abs(off.mean().item()) <= cut + 1e-5


@gpu
def test_dweight_of_the_same_tokens_again():
    """65536 tokens 16 times over: every chunk's sum is the same number P, and 16 additions of it in fp32 are
    within 16 2^-24 of 16 P.  Both are rounded to bf16, to neighbours at most, and only where 16 P is that close
    to the middle of two: 2 16 2^-24 of the 2^-8 or more between them, one in a thousand or so."""
    import torch
    D = 1536
    dy, x = tokens_of_one_sign(1 << 16, D, 14)
    w = torch.zeros(D, D, dtype=torch.bfloat16, device="cuda")
    once = ldn.linear_backward(dy, x, w, dx=False)["dweight"].double()
    got = ldn.linear_backward(dy.repeat(16, 1), x.repeat(16, 1), w, dx=False)["dweight"].double()
    off = (got - 16 * once).abs() / (16 * once)
    assert off.max().item() <= 2.0 ** -7 and (off > 0).double().mean().item() <= 2.0 ** -8


@gpu
@pytest.mark.parametrize("M,K,N,res,act,bias,save", [(40, 70400, 300, "bf16", "silu", True, True),
                                                     (300, 66000, 520, None, "gelu", True, True),
                                                     (130, 65600, 200, "bf16", None, False, False),
                                                     (2060, 66000, 1030, "bf16", None, True, True)])
def test_bf16_results_of_long_sums(M, K, N, res, act, bias, save):
    import torch
    p = linear_inputs(M, K, N, "bf16", "bf16", bias, seed=13)
    r = p["r"] if res else None
    args = dev(p["x"], "bf16"), dev(p["w"], "bf16"), dev(p["b"], "bf16"), dev(r, "bf16") if res else None
    y = ldn.linear(*args, activation=act, save_z=save)
    y, z = y if save else (y, None)
    b = ref.linear_bounds(p["x"], p["w"], p["b"], r, act, "bf16", "bf16")
    wy, wz = ref.linear(p["x"], p["w"], p["b"], r, act)
    within(y, wy, b["y"], "y")
    if save:
        within(z, wz, b["z"], "z")
    again = ldn.linear(*args, activation=act)
    assert torch.equal(again, y)


# ---- fp32 results from 8 bits, over more than one chunk ----
@gpu
@pytest.mark.parametrize("M,K,N,act", [(5, 20000, 130, None), (16, 8208, 520, "silu"), (40, 4112, 300, None),
                                       (300, 8200, 40, "gelu"), (1030, 4100, 2060, None)])
def test_linear_e4m3_long_sums(M, K, N, act):
    """A chunk of 2048 products in 8 bits is 64 additions in tensor memory, as 1024 in 16 bits are: the norm of
    what is off before the activation is within 64 steps of 2^-23 of the result's."""
    import torch
    r = np.random.default_rng(15)
    q = dev(r.normal(size=(M, K)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    wq = dev(r.normal(size=(N, K)) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    sx, sw = dev(np.exp(r.normal(size=M)) / 1e4), dev(np.exp(r.normal(size=N)) / 1e4)
    b, re = dev(r.normal(size=N), "bf16"), dev(r.normal(size=(M, N)))
    y = ldn.linear_e4m3(q, sx, wq, sw, b, re, activation=act)
    x, w = host(q.float()) * host(sx)[:, None], host(wq.float()) * host(sw)[:, None]
    want, z = ref.linear(x, w, host(b), host(re), act)
    bound = ref.linear_bounds(x, w, host(b), host(re), act, "bf16", "f32")["y"]
    within(y, want, bound + ref.SLOPE * 4 * ref.U * np.abs(z - host(b)), "y")
    if act is None:
        assert np.linalg.norm(host(y) - want) <= 64 * 2.0 ** -23 * np.linalg.norm(want)
    same = re.clone()
    assert torch.equal(ldn.linear_e4m3(q, sx, wq, sw, b, same, activation=act, out=same), y)


# ---- GELU ----
@gpu
def test_gelu_and_its_slope_to_fp32s_digits():
    """Through a product with the identity, whose z is x itself.  In steps U = 2^-24 of the tail Phi(-|z|): the
    exponential 4, and its argument 3 z^2 / 2 (z^2, its factor and their product); t = 1 / (1 + p |z|) 3, which the
    tail follows to the power of 2.4 at most; the polynomial's own sum 5 (its terms are 2.4 times the sum at most), two
    products and the fit 3: 20 + 1.5 z^2 in all, and one or two more for what follows."""
    import math

    import torch
    z = np.concatenate([np.linspace(-12, 12, 6007), [0.0, -0.0, 1e-30, -1e-30, 0.75, -0.75, 40.0, -40.0, 3e38]])
    z = np.float32(z).reshape(-1, 64)
    eye = torch.eye(64, device="cuda")
    y, got = ldn.linear(dev(z), eye, activation="gelu", save_z=True)
    assert torch.equal(got, dev(z))
    z = z.astype(np.float64)
    tail = np.vectorize(lambda v: math.erfc(abs(v) / math.sqrt(2)) / 2)(z)
    phi = np.where(z > 0, 1 - tail, tail)
    e = (20 + 1.5 * np.minimum(z * z, 200.0)) * ref.U * tail + 2.0 ** -126     # results below it are zero
    within(y, z * phi, np.abs(z) * (e + 2 * ref.U * phi), "gelu")
    with np.errstate(under="ignore"):
        bell = z * np.exp(-np.minimum(z * z, 1e4) / 2) / math.sqrt(2 * math.pi)
    g = ldn.linear_backward(torch.ones_like(y), dev(np.float32(z)), eye, got, activation="gelu")["dx"]
    bound = e + 2 * ref.U * phi + (8 + 1.5 * np.minimum(z * z, 200.0)) * ref.U * np.abs(bell) + np.abs(z) * 2.0 ** -126
    within(g, phi + bell, bound + 1.1e-38, "slope")


# ---- calls that the documentation allows ----
@gpu
@pytest.mark.parametrize("dtype,dy_dtype,act", [("bf16", "bf16", None), ("bf16", "f32", None), ("bf16", "bf16", "silu"),
                                                ("f32", "f32", None), ("f32", "f32", "gelu")])
@pytest.mark.parametrize("M,K,N,pad", [(300, 264, 520, 0), (1, 72, 130, 0), (1000, 65, 77, 3)])
def test_linear_backward_with_outputs_left_out(M, K, N, pad, dtype, dy_dtype, act):
    """Each of dx, dweight and dbias may be NULL: the others are what they are with all of them, bit for bit, on a
    workspace of exactly the size for what is wanted, between guards."""
    import torch
    p = linear_inputs(M, K, N, dtype, dy_dtype, False, seed=16)
    x, w, dy = dev(p["x"], dtype, pad=pad), dev(p["w"], dtype), dev(p["dy"], dy_dtype)
    z = dev(linear_inputs(M, K, N, dtype, dtype, False, seed=17)["r"], dtype) if act else None
    every = ldn.linear_backward(dy, x, w, z, activation=act, bias=True)
    codes = {"f32": ldn.LDN_F32, "bf16": ldn.LDN_BF16}
    how = {None: ldn.LDN_ACT_NONE, "silu": ldn.LDN_ACT_SILU, "gelu": ldn.LDN_ACT_GELU}[act]
    q = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    for want in range(8):
        out = [torch.empty_like(every[k]) if want >> i & 1 else None for i, k in enumerate(("dx", "dweight", "dbias"))]
        a = (dy.data_ptr(), x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0))
        need = ldn.ldn_linear_backward_workspace_size(*a, M, K, N, how, codes[dtype], codes[dy_dtype], want)
        guard = 1 << 18
        room = torch.full((guard + need + guard,), 0x5a, dtype=torch.uint8, device="cuda")
        st = ldn.ldn_linear_backward(*a, q(z), *map(q, out), M, K, N, how, codes[dtype], codes[dy_dtype],
                                     room.data_ptr() + guard if need else None, need,
                                     torch.cuda.current_stream().cuda_stream)
        assert st == ldn.LDN_OK
        torch.cuda.synchronize()
        assert (room[:guard] == 0x5a).all() and (room[guard + need:] == 0x5a).all()
        for k, v in zip(("dx", "dweight", "dbias"), out):
            assert v is None or torch.equal(v, every[k]), (want, k)


FIRST = """
import torch, gated_delta_rule_chunkwise_gb300 as ldn
x, w = torch.ones(40, 64, device="cuda"), torch.ones(72, 64, device="cuda")
n, m = torch.ones(72, device="cuda"), torch.zeros(40, 72, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    z = ldn.linear(x, w)
    y, s = ldn.gated_add_rmsnorm(z, m, n, n, n)
    d = ldn.gated_add_rmsnorm_backward(y, z, s, n, n, n)
    e = ldn.linear_backward(d["dx"], x, w, bias=True)
g.replay()
torch.cuda.synchronize()
assert (z == 64).all() and torch.isfinite(e["dweight"]).all()
assert (s - 1).abs().max() < 1e-5 and (y - 1).abs().max() < 1e-5 and d["dgate"].shape == (72,)
"""


@gpu
def test_first_calls_are_captured():
    """A process whose first calls are captured into a graph."""
    import os
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


@gpu
def test_calls_from_several_threads():
    import threading

    import torch
    sets = []
    for i, (M, D, H) in enumerate([(5, 256, 520), (300, 1024, 2056), (2100, 264, 1032), (64, 2048, 512)]):
        g = torch.Generator(device="cuda").manual_seed(i)
        f = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        sets.append((f(M, D).bfloat16(), (f(H, D) * D ** -0.5).bfloat16(), f(M, H), 1 + 0.1 * f(H), f(H)))

    def steps(x, w, r, n, gate):
        y = ldn.linear(x, w, None, r)
        o, s = ldn.gated_add_rmsnorm(y, r, n, n, gate, gate_sigmoid=True)
        d = ldn.gated_add_rmsnorm_backward(o, y, s, n, n, gate, r, gate_sigmoid=True)
        e = ldn.linear_backward(d["dx"], x, w, bias=True)
        return [y, o, s, *d.values(), *e.values()]
    want = [steps(*s) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = steps(*sets[i])
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)
        except Exception as e:  # a thread's own is lost
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are what they are alone (each row's norm is its own), and a
    projection's last rows what plain fp32 products give, to bf16's rounding (2^-8) and what fp32 sums of 64 or
    16384 products of a size of 1 and a row's norm of 1 or 16 leave (6e-8 and 2e-5 of it)."""
    import torch
    D, rows, last = 16384, (1 << 17) + 900, 400
    x = torch.randn(last, D, device="cuda").bfloat16().repeat(-(-rows // last), 1)[:rows]
    r, n = x.flip(1), 1 + 0.1 * torch.randn(D, device="cuda")
    assert rows * D > 1 << 31
    y, s = ldn.gated_add_rmsnorm(x, r, n, n, x, gate_sigmoid=True)
    g = ldn.gated_add_rmsnorm_backward(x, x, s, n, n, x, r, gate_sigmoid=True)
    tail = lambda t: t[-last:].contiguous()  # noqa: E731
    y2, s2 = ldn.gated_add_rmsnorm(tail(x), tail(r), n, n, tail(x), gate_sigmoid=True)
    g2 = ldn.gated_add_rmsnorm_backward(tail(x), tail(x), s2, n, n, tail(x), tail(r), gate_sigmoid=True)
    assert torch.equal(tail(y), y2) and torch.equal(tail(s), s2)
    assert all(torch.equal(tail(g[k]), g2[k]) for k in ("dx", "dresidual", "dgate"))
    del y, s, g, r
    w = (torch.randn(64, D, device="cuda") / 128).bfloat16()
    wide = x[:, :64]                                    # rows 16384 apart
    for a, b in ((x, w), (wide, w[:, :64]), (wide, (torch.randn(D, 64, device="cuda") / 8).bfloat16())):
        y = ldn.linear(a, b, activation="silu")
        own = torch.nn.functional.silu(a[-last:].float() @ b.float().t())
        assert ((y[-last:].float() - own).abs() <= 2.0 ** -8 * own.abs() + 1e-4).all()
    # y is [rows][16384] now: its gradients
    g = ldn.linear_backward(y, wide, b, bias=True)
    own = y[-last:].float() @ b.float()
    assert ((g["dx"][-last:].float() - own).abs() <= 2.0 ** -8 * own.abs() + 1e-3).all()
    want = sum(p.sum(0, dtype=torch.float64) for p in y.split(1 << 14))
    # rounding of the result, and of at most rows / 256 + 256 sums of a column in fp32
    size = sum(p.float().abs().sum(0, dtype=torch.float64) for p in y.split(1 << 14))
    assert ((g["dbias"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 800 * 2.0 ** -24 * size).all()
