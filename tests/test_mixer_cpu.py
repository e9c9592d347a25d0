"""Host side of the operators around a token mixer: refusals of the C entry points (before
any CUDA call), workspace sizes, the torch layer's checks, and the 64-bit references'
gradients against differences."""
import numpy as np
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from gated_delta_rule_chunkwise_gb300 import build as ldn_build
from tests import _mixer_ref as ref

BAD, UNSUP, OK = ldn.LDN_ERR_INVALID_ARG, ldn.LDN_ERR_UNSUPPORTED, ldn.LDN_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    ldn_build.build()
    return ldn.load()


def at(i):
    """Addresses far apart, 256-byte aligned, never read."""
    return (i + 1) << 32


# ---- refusals ----
NORM = dict(x=at(0), residual=at(1), weight=at(2), y=at(3), residual_out=at(4), rows=3, D=64, dtype=1,
            residual_dtype=1, eps=1e-6, stream=None)
NORM_BAD = [(dict(x=None), BAD), (dict(weight=None), BAD), (dict(y=None), BAD), (dict(residual_out=None), BAD),
            (dict(residual=None), BAD), (dict(rows=-1), BAD), (dict(D=0), BAD), (dict(dtype=2), BAD),
            (dict(residual_dtype=5), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
            (dict(D=32769), UNSUP), (dict(dtype=0, residual_dtype=1), UNSUP), (dict(rows=1 << 31), UNSUP),
            (dict(x=at(0) + 1), BAD), (dict(weight=at(2) + 2), BAD), (dict(residual=at(1) + 1), BAD),
            (dict(y=at(0)), BAD), (dict(y=at(1)), BAD), (dict(residual_out=at(0)), BAD),
            (dict(residual_out=at(1) + 64), BAD), (dict(residual_out=at(3) + 128), BAD), (dict(rows=0, x=None), OK)]


@pytest.mark.parametrize("kw,want", NORM_BAD)
def test_add_rmsnorm_refuses(kw, want):
    a = NORM | kw
    assert ldn.ldn_add_rmsnorm(*a.values()) == want


E4M3 = dict(x=at(0), residual=at(1), weight=at(2), q=at(3), scale=at(5), residual_out=at(4), rows=3, D=64, group=0,
            dtype=1, residual_dtype=1, eps=1e-6, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(scale=None), BAD), (dict(q=None), BAD), (dict(group=64), UNSUP),
                                     (dict(group=-128), UNSUP), (dict(scale=at(5) + 2), BAD), (dict(scale=at(3)), BAD),
                                     (dict(D=0), BAD), (dict(rows=0), OK)])
def test_add_rmsnorm_e4m3_refuses(kw, want):
    a = E4M3 | kw
    assert ldn.ldn_add_rmsnorm_e4m3(*a.values()) == want


NORMB = dict(dy=at(0), s=at(1), weight=at(2), dsum=at(3), dx=at(4), dresidual=at(5), dweight=at(6), rows=3, D=64,
             dtype=1, residual_dtype=0, eps=1e-6, workspace=at(7), workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(dy=None), BAD), (dict(s=None), BAD), (dict(dweight=None), BAD),
                                     (dict(workspace=None), BAD), (dict(workspace_bytes=100), BAD),
                                     (dict(workspace=at(7) + 4), BAD), (dict(dx=at(0)), BAD), (dict(dx=at(3)), BAD),
                                     (dict(dresidual=at(4)), BAD), (dict(dtype=7), BAD), (dict(eps=-1.0), BAD),
                                     (dict(D=40000), UNSUP), (dict(dtype=0, residual_dtype=1), UNSUP),
                                     (dict(dsum=at(3) + 2), BAD), (dict(dweight=at(7) + 16), BAD)])
def test_add_rmsnorm_backward_refuses(kw, want):
    a = NORMB | kw
    assert ldn.ldn_add_rmsnorm_backward(*a.values()) == want


CONV = dict(x=at(0), ldx=64, weight=at(1), bias=at(2), state=at(3), lens=at(4), y=at(5), state_out=at(6), B=2, T=9,
            C=64, width=4, activation=1, dtype=1, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(x=None), BAD), (dict(weight=None), BAD), (dict(y=None), BAD),
                                     (dict(ldx=63), BAD), (dict(B=0), BAD), (dict(T=-1), BAD), (dict(C=0), BAD),
                                     (dict(width=0), BAD), (dict(width=9), UNSUP), (dict(activation=2), BAD),
                                     (dict(dtype=3), BAD), (dict(x=at(0) + 1), BAD), (dict(lens=at(4) + 2), BAD),
                                     (dict(y=at(0)), BAD), (dict(state_out=at(5)), BAD), (dict(y=at(3)), BAD),
                                     (dict(state_out=at(3) + 128), BAD), (dict(ldx=1 << 41), UNSUP),
                                     (dict(T=0, state_out=None), OK)])
def test_short_conv_refuses(kw, want):
    a = CONV | kw
    assert ldn.ldn_short_conv(*a.values()) == want


CSTEP = dict(x=at(0), ldx=64, weight=at(1), bias=at(2), state=at(3), y=at(5), state_out=at(3), B=2, C=64, width=4,
             activation=1, dtype=1, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(x=None), BAD), (dict(state=None), BAD), (dict(state_out=None), BAD),
                                     (dict(y=at(3)), BAD), (dict(width=9), UNSUP), (dict(ldx=8), BAD),
                                     (dict(state_out=at(3) + 128), BAD), (dict(y=at(0)), BAD)])
def test_short_conv_step_refuses(kw, want):
    a = CSTEP | kw
    assert ldn.ldn_short_conv_step(*a.values()) == want


CBWD = dict(x=at(0), ldx=64, weight=at(1), bias=at(2), state=at(3), lens=at(4), dy=at(5), dstate_out=at(6), dx=at(7),
            dweight=at(8), dbias=at(9), dstate=at(10), B=2, T=9, C=64, width=4, activation=1, dtype=1,
            workspace=at(11), workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(dy=None), BAD), (dict(dx=None), BAD), (dict(dweight=None), BAD),
                                     (dict(workspace=None), BAD), (dict(workspace_bytes=16), BAD),
                                     (dict(dx=at(5)), BAD), (dict(dx=at(0)), BAD), (dict(dstate=at(3)), BAD),
                                     (dict(dbias=at(9) + 2), BAD), (dict(width=9), UNSUP), (dict(T=-1), BAD)])
def test_short_conv_backward_refuses(kw, want):
    a = CBWD | kw
    assert ldn.ldn_short_conv_backward(*a.values()) == want


SCAN = dict(u=at(0), ldu=64, delta=at(1), ld_delta=64, A=at(2), Bm=at(3), ldb=32, Cm=at(4), ldc=32, Dskip=at(5),
            z=at(6), ldz=64, delta_bias=at(7), h0=at(8), lens=at(9), y=at(10), h_final=at(11), states=at(12), B=2,
            T=40, D=64, N=16, G=2, delta_softplus=1, dtype=1, workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(u=None), BAD), (dict(delta=None), BAD), (dict(A=None), BAD),
                                     (dict(Bm=None), BAD), (dict(Cm=None), BAD), (dict(y=None), BAD),
                                     (dict(ldu=63), BAD), (dict(ldb=31), BAD), (dict(ldc=0), BAD), (dict(ldz=1), BAD),
                                     (dict(N=0), BAD), (dict(N=24), UNSUP), (dict(G=0), BAD), (dict(G=3), BAD),
                                     (dict(B=0), BAD), (dict(T=-1), BAD), (dict(dtype=2), BAD),
                                     (dict(delta_softplus=2), BAD), (dict(h0=at(8) + 4), BAD),
                                     (dict(states=at(12) + 8), BAD), (dict(h_final=at(8)), BAD), (dict(y=at(0)), BAD),
                                     (dict(y=at(6)), BAD), (dict(states=at(11)), BAD), (dict(A=at(2) + 2), BAD),
                                     (dict(T=0, h_final=None), OK)])
def test_ssm_scan_refuses(kw, want):
    a = SCAN | kw
    assert ldn.ldn_ssm_scan(*a.values()) == want


STEP = dict(u=at(0), ldu=64, delta=at(1), ld_delta=64, A=at(2), Bm=at(3), ldb=32, Cm=at(4), ldc=32, Dskip=at(5),
            z=at(6), ldz=64, delta_bias=at(7), h=at(8), h_out=at(8), y=at(10), B=2, D=64, N=16, G=2,
            delta_softplus=1, dtype=1, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(h=None), BAD), (dict(h_out=None), BAD), (dict(y=at(8)), BAD),
                                     (dict(h_out=at(8) + 16), BAD), (dict(N=12), UNSUP), (dict(ldu=1), BAD),
                                     (dict(z=at(6) + 1), BAD), (dict(u=None), BAD)])
def test_ssm_step_refuses(kw, want):
    a = STEP | kw
    assert ldn.ldn_ssm_step(*a.values()) == want


SBWD = dict(u=at(0), ldu=64, delta=at(1), ld_delta=64, A=at(2), Bm=at(3), ldb=32, Cm=at(4), ldc=32, Dskip=at(5),
            z=at(6), ldz=64, delta_bias=at(7), states=at(8), lens=at(9), dy=at(10), dh_final=at(11), du=at(12),
            ddelta=at(13), dA=at(14), dB=at(15), dC=at(16), dD=at(17), dz=at(18), ddelta_bias=at(19), dh0=at(20), B=2,
            T=40, D=64, N=16, G=2, delta_softplus=1, dtype=1, workspace=at(21), workspace_bytes=1 << 31, stream=None)


@pytest.mark.parametrize("kw,want", [(dict(states=None), BAD), (dict(dy=None), BAD), (dict(dA=None), BAD),
                                     (dict(dz=None), BAD), (dict(z=None), BAD), (dict(workspace=None), BAD),
                                     (dict(workspace_bytes=1024), BAD), (dict(du=at(10)), BAD), (dict(dB=at(16)), BAD),
                                     (dict(dh0=at(20) + 4), BAD), (dict(N=5), UNSUP), (dict(G=5), BAD),
                                     (dict(dh0=at(11)), BAD), (dict(dC=None), BAD)])
def test_ssm_backward_refuses(kw, want):
    a = SBWD | kw
    assert ldn.ldn_ssm_backward(*a.values()) == want


# ---- workspaces ----
def test_workspace_sizes():
    assert ldn.ldn_add_rmsnorm_backward_workspace_size(0, 64) == 0
    assert ldn.ldn_add_rmsnorm_backward_workspace_size(5, 64) == 5 * 64 * 4       # a block a row
    assert ldn.ldn_add_rmsnorm_backward_workspace_size(5, 0) == 0
    assert ldn.ldn_short_conv_backward_workspace_size(1, 5, 64, 9) == 0
    assert ldn.ldn_short_conv_backward_workspace_size(3, 1, 64, 4) == 3 * 5 * 64 * 4
    assert ldn.ldn_ssm_scan_workspace_size(1, 64, 4096, 16, 1) == 0               # too short to cut
    assert ldn.ldn_ssm_scan_workspace_size(1, 65536, 64, 16, 1) > 0
    assert ldn.ldn_ssm_scan_workspace_size(1, 64, 64, 17, 1) == 0
    assert ldn.ldn_ssm_backward_workspace_size(1, 0, 64, 16, 1) == 0
    assert ldn.ldn_ssm_backward_workspace_size(1, 1, 64, 16, 1) > 0


# ---- the torch layer ----
def test_torch_layer_wants_cuda_tensors():
    import torch
    x = torch.zeros(2, 8)
    w = torch.ones(8)
    with pytest.raises(TypeError):
        ldn.add_rmsnorm(x, None, w)
    with pytest.raises(TypeError):
        ldn.short_conv_step(x, torch.ones(8, 4), None, torch.zeros(2, 3, 8))
    with pytest.raises(TypeError):
        ldn.selective_scan_step(x, x, w, x, x, None, None, None, x)


def test_row_distances_of_views():
    """The distance between rows that views have, and the views that have none."""
    import torch
    from gated_delta_rule_chunkwise_gb300 import mixer
    f = mixer._core.row_distance
    x = torch.zeros(3, 5, 16)
    assert f(x, 2) == 16
    assert f(x[:, :, 4:12], 2) == 16
    assert f(x[:1, :, 4:12], 2) == 16
    assert f(x[:, :1, 4:12], 2) == 80
    assert f(x[:1, :1, 4:12], 2) == 8
    assert f(x[:, 2, 4:12], 1) == 80
    b = torch.zeros(3, 5, 40)[..., 3:35].unflatten(-1, (2, 16))
    assert f(b, 2) == 40
    for bad in (x[:, ::2, :], x[:, 1:4, :], x.transpose(0, 1), x.transpose(1, 2), x[..., ::2],
                x[:, :1, :].expand(3, 5, 16)):
        assert f(bad, 2) == -1


# ---- the references' gradients against differences ----
def _check(f, args, grads, h=1e-5):
    rng = np.random.default_rng(0)
    for name, g in grads.items():
        a = args[name]
        for _ in range(6):
            at_ = tuple(rng.integers(0, n) for n in a.shape)
            keep = a[at_]
            a[at_] = keep + h
            up = f()
            a[at_] = keep - h
            down = f()
            a[at_] = keep
            # central differences: h^2 times a third derivative of order one, and rounding / h
            assert abs((up - down) / (2 * h) - g[at_]) < 1e-6 * (1 + abs(g[at_])), name


def test_reference_gradients_norm():
    r = np.random.default_rng(1)
    a = dict(s=r.normal(size=(3, 10)), w=r.normal(size=10))
    dy, dsum = r.normal(size=(3, 10)), r.normal(size=(3, 10))
    ds, dw = ref.norm_bwd(dy, a["s"], a["w"], dsum, 1e-3)
    _check(lambda: (dy * ref.norm(a["s"], a["w"], 1e-3)).sum() + (dsum * a["s"]).sum(), a, dict(s=ds, w=dw))


@pytest.mark.parametrize("act", [True, False])
def test_reference_gradients_conv(act):
    r = np.random.default_rng(2)
    lens = [7, 2, 0]
    a = dict(x=r.normal(size=(3, 7, 5)), w=r.normal(size=(5, 4)), b=r.normal(size=5), st=r.normal(size=(3, 3, 5)))
    dy, dl = r.normal(size=(3, 7, 5)), r.normal(size=(3, 3, 5))

    def loss():
        y, _, last = ref.conv(a["x"], a["w"], a["b"], a["st"], lens, act)
        return (dy * y).sum() + (dl * last).sum()
    dx, dw, db, dst = ref.conv_bwd(a["x"], a["w"], a["b"], a["st"], lens, act, dy, dl)
    _check(loss, a, dict(x=dx, w=dw, b=db, st=dst))


@pytest.mark.parametrize("gate", [True, False])
def test_reference_gradients_scan(gate):
    r = np.random.default_rng(3)
    B, T, D, G, N, lens = 2, 6, 4, 2, 3, [6, 4]
    p = dict(u=r.normal(size=(B, T, D)), delta=r.normal(size=(B, T, D)), A=-np.abs(r.normal(size=(D, N))),
             B=r.normal(size=(B, T, G, N)), C=r.normal(size=(B, T, G, N)), D=r.normal(size=D),
             z=r.normal(size=(B, T, D)) if gate else None, bias=r.normal(size=D), h0=r.normal(size=(B, D, N)),
             softplus=gate)
    dy, dh = r.normal(size=(B, T, D)), r.normal(size=(B, D, N))

    def loss():
        y, h = ref.scan(p, lens)[:2]
        return (dy * y).sum() + (dh * h[:, -1]).sum()
    g = ref.scan_bwd(p, lens, dy, dh)
    names = dict(u="du", delta="ddelta", A="dA", B="dB", C="dC", D="dD", bias="ddelta_bias", h0="dh0")
    if gate:
        names["z"] = "dz"
    _check(loss, p, {k: g[v] for k, v in names.items()})


def test_e4m3_reference():
    import torch
    v = np.concatenate([np.linspace(-500, 500, 4001), np.linspace(-0.05, 0.05, 1001), [0.0, 464.0, -480.0]])
    # what lies past the largest value saturates in the kernel; torch's own cast gives NaN there
    got = torch.from_numpy(np.clip(v, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(np.clip(v, -448, 448).astype(np.float32).astype(np.float64)), got)


def test_sequences_near_the_largest_int_are_refused():
    """Runs and segments of tokens may end a little past the sequence, so a length within
    2^16 of the largest int is refused."""
    most = (1 << 31) - 1 - (1 << 16)
    for T, st in ((most, True), (most + 1, False), ((1 << 31) - 1, False)):
        assert (ldn.ldn_short_conv_backward_workspace_size(1, T, 1, 4) > 0) == st
        assert (ldn.ldn_ssm_backward_workspace_size(1, T, 16, 8, 1) > 0) == st
