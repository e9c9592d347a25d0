"""Host side of the operators that join blocks: refusals of the C entry points (before any CUDA
call), workspace sizes, the plans of the products, and the 64-bit references' gradients against
differences."""
import os
import subprocess

import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from gated_delta_rule_chunkwise_gb300 import build as ldn_build
from tests import _join_ref as ref
from tests.test_mixer_cpu import _check, at

BAD, UNSUP, OK = ldn.LDN_ERR_INVALID_ARG, ldn.LDN_ERR_UNSUPPORTED, ldn.LDN_OK
MOST = (1 << 31) - 1 - (1 << 16)


@pytest.fixture(scope="module", autouse=True)
def lib():
    ldn_build.build()
    return ldn.load()


# ---- refusals ----
GATED = dict(x=at(0), residual=at(1), gate=at(2), post_weight=at(3), weight=at(4), y=at(5), residual_out=at(6), rows=6,
             D=64, gate_rows=3, gate_dtype=1, gate_sigmoid=0, residual_scale=1.0, dtype=1, residual_dtype=0, eps=1e-6,
             stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(residual=None), BAD), (dict(residual_out=None), BAD), (dict(y=None), BAD),
    (dict(weight=None), BAD), (dict(rows=-1), BAD), (dict(D=0), BAD), (dict(gate_rows=4), BAD),
    (dict(gate_rows=0), BAD), (dict(gate_rows=-3), BAD), (dict(gate_rows=12), BAD), (dict(gate_dtype=2), BAD),
    (dict(gate_sigmoid=2), BAD), (dict(residual_scale=float("inf")), BAD), (dict(residual_scale=float("nan")), BAD),
    (dict(dtype=5), BAD), (dict(residual_dtype=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(dtype=0, gate_dtype=1), UNSUP), (dict(dtype=0, gate_dtype=0, residual_dtype=1), UNSUP),
    (dict(D=16385), UNSUP), (dict(rows=3 << 30), UNSUP), (dict(x=at(0) + 1), BAD), (dict(gate=at(2) + 1), BAD),
    (dict(weight=at(4) + 2), BAD), (dict(residual=at(1) + 2), BAD), (dict(y=at(0)), BAD), (dict(y=at(2)), BAD),
    (dict(residual_out=at(1) + 64), BAD), (dict(residual_out=at(5)), BAD), (dict(residual_out=at(0)), BAD),
    (dict(rows=0, x=None), OK), (dict(rows=0, gate_rows=0), OK)])
def test_gated_add_rmsnorm_refuses(kw, want):
    assert ldn.ldn_gated_add_rmsnorm(*(GATED | kw).values()) == want


GATEDB = dict(dy=at(0), x=at(1), s=at(2), dsum=at(3), gate=at(4), post_weight=at(5), weight=at(6), dx=at(7),
              dresidual=at(8), dgate=at(9), dpost_weight=at(10), dweight=at(11), rows=6, D=64, gate_rows=3,
              gate_dtype=1, gate_sigmoid=0, residual_scale=1.0, dtype=1, residual_dtype=0, eps=1e-6, workspace=at(12),
              workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), BAD), (dict(x=None), BAD), (dict(s=None), BAD), (dict(weight=None), BAD), (dict(dweight=None), BAD),
    (dict(post_weight=None), BAD), (dict(dpost_weight=None), BAD), (dict(gate=None), BAD), (dict(gate_rows=4), BAD),
    (dict(workspace=None), BAD), (dict(workspace_bytes=16), BAD), (dict(workspace=at(12) + 8), BAD),
    (dict(dx=at(0)), BAD), (dict(dresidual=at(3)), BAD), (dict(dgate=at(4)), BAD), (dict(dgate=at(9) + 1), BAD),
    (dict(dweight=at(10) + 64), BAD), (dict(dweight=at(12) + 64), BAD), (dict(D=16385), UNSUP),
    (dict(dtype=0, gate_dtype=0, residual_dtype=1), UNSUP), (dict(eps=-1.0), BAD), (dict(gate_sigmoid=-1), BAD)])
def test_gated_add_rmsnorm_backward_refuses(kw, want):
    assert ldn.ldn_gated_add_rmsnorm_backward(*(GATEDB | kw).values()) == want


def test_gated_workspace_sizes():
    f = ldn.ldn_gated_add_rmsnorm_backward_workspace_size
    assert f(0, 64, 0) == 0 and f(4, 0, 0) == 0 and f(4, 16385, 0) == 0 and f(6, 64, 4) == 0 and f(6, 64, -1) == 0
    # two shares of columns a block, and a gate's row of each run of rows that shares it
    assert f(1, 64, 0) == 2 * 64 * 4 and f(1, 64, 1) == 2 * 64 * 4
    for rows, gates in ((6, 3), (4096, 1), (4096, 2), (4096, 512), (4096, 2048), (7 * 1111, 7)):
        assert f(rows, 64, gates) >= (2 + gates) * 64 * 4


LIN = dict(x=at(0), ldx=64, weight=at(1), ldw=64, bias=at(2), residual=at(3), y=at(4), z=at(5), rows=5, K=64, N=40,
           activation=1, dtype=1, out_dtype=1, workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(weight=None), BAD), (dict(y=None), BAD), (dict(ldx=63), BAD), (dict(ldw=8), BAD),
    (dict(rows=-1), BAD), (dict(K=0), BAD), (dict(N=0), BAD), (dict(activation=3), BAD), (dict(activation=-1), BAD),
    (dict(dtype=2), BAD), (dict(out_dtype=7), BAD), (dict(dtype=0, out_dtype=1), UNSUP), (dict(x=at(0) + 1), BAD),
    (dict(weight=at(1) + 1), BAD), (dict(bias=at(2) + 1), BAD), (dict(residual=at(3) + 1), BAD), (dict(y=at(4) + 1), BAD),
    (dict(z=at(5) + 1), BAD), (dict(y=at(0)), BAD), (dict(y=at(1)), BAD), (dict(z=at(4)), BAD), (dict(z=at(3)), BAD),
    (dict(y=at(3) + 16), BAD), (dict(y=at(2)), BAD),
    # rows that do not start at 16-byte boundaries, and fp32, need room to be laid out
    (dict(ldx=65), BAD), (dict(ldw=66), BAD), (dict(x=at(0) + 2), BAD), (dict(K=63, ldx=63), BAD),
    (dict(dtype=0, out_dtype=0), BAD), (dict(ldx=65, workspace=at(6) + 16, workspace_bytes=1 << 20), BAD),
    (dict(ldx=65, workspace=at(6), workspace_bytes=128), BAD), (dict(ldx=65, workspace=at(4), workspace_bytes=1 << 20), BAD),
    (dict(rows=MOST + 1), UNSUP), (dict(K=MOST + 1, ldx=1 << 31, ldw=1 << 31), UNSUP), (dict(N=MOST + 1), UNSUP),
    (dict(ldx=1 << 39), UNSUP), (dict(rows=MOST, ldx=1 << 12), UNSUP), (dict(rows=0, x=None, y=None), OK)])
def test_linear_refuses(kw, want):
    assert ldn.ldn_linear(*(LIN | kw).values()) == want


E4M3 = dict(x=at(0), ldx=64, x_scale=at(6), weight=at(1), ldw=64, weight_scale=at(7), bias=at(2), residual=at(3),
            y=at(4), rows=5, K=64, N=40, activation=0, out_dtype=1, workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x_scale=None), BAD), (dict(weight_scale=None), BAD), (dict(x=None), BAD), (dict(y=at(6)), BAD),
    (dict(x_scale=at(6) + 2), BAD), (dict(weight_scale=at(7) + 1), BAD), (dict(ldx=72), BAD), (dict(x=at(0) + 8), BAD),
    (dict(K=60, ldx=60), BAD), (dict(out_dtype=2), BAD), (dict(activation=4), BAD), (dict(rows=0), OK)])
def test_linear_e4m3_refuses(kw, want):
    assert ldn.ldn_linear_e4m3(*(E4M3 | kw).values()) == want


LINB = dict(dy=at(0), x=at(1), ldx=64, weight=at(2), ldw=64, z=at(3), dx=at(4), dweight=at(5), dbias=at(6), rows=5,
            K=64, N=40, activation=1, dtype=1, dy_dtype=1, workspace=at(7), workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), BAD), (dict(x=None), BAD), (dict(weight=None), BAD), (dict(z=None), BAD), (dict(workspace=None), BAD),
    (dict(workspace_bytes=16), BAD), (dict(workspace=at(7) + 64), BAD), (dict(ldx=1), BAD), (dict(ldw=63), BAD),
    (dict(activation=3), BAD), (dict(dtype=3), BAD), (dict(dy_dtype=3), BAD), (dict(dtype=0, dy_dtype=1), UNSUP),
    (dict(dx=at(0)), BAD), (dict(dweight=at(1)), BAD), (dict(dbias=at(5)), BAD), (dict(dx=at(3)), BAD),
    (dict(dweight=at(7)), BAD), (dict(dx=at(4) + 1), BAD), (dict(N=MOST + 1), UNSUP)])
def test_linear_backward_refuses(kw, want):
    assert ldn.ldn_linear_backward(*(LINB | kw).values()) == want


def test_linear_workspace_sizes():
    f = ldn.ldn_linear_workspace_size
    assert f(at(0), 64, at(1), 64, 5, 64, 40, 1) == 0                       # bf16, as it lies in memory
    assert f(at(0) + 2, 64, at(1), 64, 5, 64, 40, 1) == 768                 # 5 rows of 64, to 256 bytes
    assert f(at(0), 65, at(1), 64, 1, 64, 40, 1) == 0                       # one row has no next one
    assert f(at(0), 63, at(1), 63, 5, 63, 40, 1) == 768 + 5120
    assert f(at(0), 64, at(1), 64, 5, 64, 40, 0) == 4 * (5 + 40) * 128      # four planes of each operand
    assert f(at(0), 64, at(1), 64, 0, 64, 40, 0) == 0 and f(at(0), 64, at(1), 63, 5, 64, 40, 0) == 0
    e = ldn.ldn_linear_e4m3_workspace_size
    assert e(at(0), 64, at(1), 64, 5, 64, 40) == 0 and e(at(0), 72, at(1), 64, 5, 64, 40) == 512
    g = ldn.ldn_linear_backward_workspace_size
    a = (at(0), at(1), 64, at(2), 64, 5, 64, 40)
    assert g(*a, 0, 1, 1, 3) == 0 and g(*a, 0, 1, 1, 7) == 256              # dz is dy; the bias's shares
    assert g(*a, 1, 1, 1, 3) == 512 and g(*a, 0, 1, 0, 1) == 512            # dz is formed: 5 rows of 40
    assert g(*a, 0, 1, 0, 4) == 256 and g(*a, 0, 1, 1, 0) == 0


def test_plans_fill_their_tiles(tmp_path):
    """Every plan takes all columns, splits no further than there are k blocks or blocks that run
    together, and gives each half of a split block's share a column at least."""
    csrc = ldn_build.CSRC
    src = tmp_path / "plan.cpp"
    src.write_text('#include <cstdio>\n#include "linear_plan.h"\nint main(){ long long i, j; int k, p, n, r;\n'
                   'while (scanf("%lld %lld %d %d %d %d", &i, &j, &k, &p, &n, &r) == 6) {\n'
                   'ldn::linear::Plan q = ldn::linear::plan_for(i, j, k, p, n, r, 152);\n'
                   'printf("%d %d %d\\n", q.bn, q.split, q.pair); } }\n')
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", exe], check=True)
    r = np.random.default_rng(0)
    cases = [(int(np.exp(r.uniform(0, np.log(20000)))), int(np.exp(r.uniform(0, np.log(20000)))),
              int(np.exp(r.uniform(0, np.log(300)))), int(r.choice([1, 6])), int(r.integers(2)), int(r.integers(2))) for _ in range(3000)]
    cases += [(1, 1, 1, 1, 0, 0), (MOST, 1, 1, 1, 0, 1), (1, MOST, 1, 1, 1, 0), (1, 1, 1 << 25, 6, 0, 1)]
    out = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True,
                         check=True).stdout.split()
    assert len(out) == 3 * len(cases)
    for (i, j, k, p, mn, promote), bn, split, pair in zip(cases, *(map(int, out[q::3]) for q in range(3))):
        assert 16 <= bn <= 256 and bn % (64 if mn else 32 if bn > 16 else 16) == 0 and split in (1, 2, 4, 8)
        stage = 128 * (128 + (bn // 2 if pair else bn))
        parts = bn * 512 if split > 1 else 0
        assert not promote or bn <= (256 if pair else 128)                  # sums that fit a thread's registers
        assert stage % 1024 == 0 and 3 <= (200 * 1024 - parts) // stage     # a ring beside the parts
        if split > 1:
            assert not pair and split <= k and -(-i // 128) * -(-j // bn) * split <= 152 and bn % (2 * split) == 0
        if pair:
            assert bn % (128 if mn else 32) == 0


# ---- the references' gradients ----
@pytest.mark.parametrize("gate,sig,post,pre", [("none", False, True, True), ("channel", True, True, True),
                                               ("sequence", False, True, False), ("token", True, False, True)])
def test_reference_gradients_gated(gate, sig, post, pre):
    r = np.random.default_rng(4)
    B, T, D = 2, 3, 8
    shape = {"none": None, "channel": (D,), "sequence": (B, 1, D), "token": (B, T, D)}[gate]
    a = dict(x=r.normal(size=(B, T, D)), r=r.normal(size=(B, T, D)))
    a |= dict(w=r.normal(size=D)) if pre else {}
    a |= dict(wp=r.normal(size=D)) if post else {}
    a |= dict(gate=r.normal(size=shape)) if shape else {}
    dy, dsum = r.normal(size=(B, T, D)), r.normal(size=(B, T, D))
    g = lambda k: a.get(k)  # noqa: E731

    def loss():
        s, y = ref.gated(a["x"], a["r"], g("w"), g("wp"), g("gate"), 0.5, sig, 1e-3)
        return (dsum * s).sum() + (0 if y is None else (dy * y).sum())
    s, _ = ref.gated(a["x"], a["r"], g("w"), g("wp"), g("gate"), 0.5, sig, 1e-3)
    got = ref.gated_bwd(dy, a["x"], s, g("w"), g("wp"), g("gate"), dsum, 0.5, sig, 1e-3)
    names = dict(x="dx", r="dresidual", w="dweight", wp="dpost_weight", gate="dgate")
    _check(loss, a, {k: got[names[k]] for k in a})


@pytest.mark.parametrize("name", [None, "silu", "gelu"])
def test_reference_gradients_linear(name):
    r = np.random.default_rng(5)
    a = dict(x=r.normal(size=(4, 5)), w=r.normal(size=(3, 5)), b=r.normal(size=3), r=r.normal(size=(4, 3)))
    dy = r.normal(size=(4, 3))
    z = ref.linear(a["x"], a["w"], a["b"], a["r"], name)[1]
    g, _ = ref.linear_bwd(dy, a["x"], a["w"], z, name)
    _check(lambda: (dy * ref.linear(a["x"], a["w"], a["b"], a["r"], name)[0]).sum(), a,
           dict(x=g["dx"], w=g["dweight"], b=g["dbias"], r=dy))


def test_the_package_names_them():
    import torch  # noqa: F401
    for n in ("gated_add_rmsnorm", "gated_add_rmsnorm_backward", "linear", "linear_backward", "linear_e4m3"):
        assert callable(getattr(ldn, n))
    assert os.path.exists(ldn_build.TORCH_LIB_PATH)
