"""Host side of the operators around a token mixer: what is refused near the largest int, and
what needs no torch or no compiler for it."""
import pytest

import gated_delta_rule_chunkwise_gb300 as ldn
from gated_delta_rule_chunkwise_gb300 import build as ldn_build
from tests.test_mixer_cpu import CBWD, CONV, CSTEP, SBWD, SCAN, STEP, UNSUP, at  # noqa: F401

MOST = (1 << 31) - 1 - (1 << 16)


@pytest.fixture(scope="module", autouse=True)
def lib():
    ldn_build.build()
    return ldn.load()


def test_channels_near_the_largest_int_are_refused():
    """Blocks of channels may end a little past the last one, so a count within 2^16 of the
    largest int is refused, as a sequence's length is."""
    for C, ok in ((MOST, True), (MOST + 1, False), ((1 << 31) - 1, False)):
        assert (ldn.ldn_short_conv_backward_workspace_size(1, 1, C, 4) > 0) == ok
        assert (ldn.ldn_ssm_backward_workspace_size(1, 1, C, 8, 1) > 0) == ok
    C = (1 << 31) - 1
    far = dict(B=1, C=C, ldx=C)
    assert ldn.ldn_short_conv(*(CONV | far | dict(T=1)).values()) == UNSUP
    assert ldn.ldn_short_conv_step(*(CSTEP | far).values()) == UNSUP
    assert ldn.ldn_short_conv_backward(*(CBWD | far | dict(T=1)).values()) == UNSUP
    far = dict(B=1, D=C, G=1, N=8, ldu=C, ld_delta=C, ldz=C)
    assert ldn.ldn_ssm_scan(*(SCAN | far | dict(T=1)).values()) == UNSUP
    assert ldn.ldn_ssm_step(*(STEP | far).values()) == UNSUP
    assert ldn.ldn_ssm_backward(*(SBWD | far | dict(T=1)).values()) == UNSUP


# ---- what needs no native torch layer ----
def in_a_process(code):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


def test_delta_rule_needs_no_native_torch_layer():
    """autograd.delta_rule runs on libldn.so alone; the operators of the native torch layer say
    what is missing where they are called."""
    in_a_process("""
import sys
sys.modules["gated_delta_rule_chunkwise_gb300.mixer"] = None    # as if its library could not be loaded
from gated_delta_rule_chunkwise_gb300 import autograd
assert callable(autograd.delta_rule)
try:
    autograd.short_conv(None, None)
except ImportError:
    pass
else:
    raise SystemExit("no ImportError")
""")


@pytest.fixture
def made(monkeypatch, tmp_path):
    """build() into an empty folder with its compilers replaced: the list of what they made."""
    import os
    done = []

    def make(path):
        with open(path, "w"):
            pass
        done.append(os.path.basename(path))
        return path

    for k in ("OBJ_DIR", "LIB_DIR"):
        monkeypatch.setattr(ldn_build, k, str(tmp_path))
    for k in ("LIB_PATH", "DIAG_LIB_PATH", "TORCH_LIB_PATH"):
        monkeypatch.setattr(ldn_build, k, str(tmp_path / os.path.basename(getattr(ldn_build, k))))
    monkeypatch.setattr(ldn_build, "_compile", lambda nvcc, src, log: src)
    monkeypatch.setattr(ldn_build, "_link", lambda nvcc, objs, path: make(path))
    monkeypatch.setattr(ldn_build, "_compile_torch", lambda log: "binding.o")
    monkeypatch.setattr(ldn_build, "_link_torch", lambda obj: make(ldn_build.TORCH_LIB_PATH))
    return done


def test_the_c_library_builds_without_torch(made, monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "torch", None)     # importing it raises ImportError
    assert ldn_build.build() == ldn_build.LIB_PATH
    assert made == ["libldn.so", "libldn_diag.so"]
    ldn_build.build()
    assert len(made) == 2


def test_the_c_library_is_in_place_where_the_torch_layer_fails(made, monkeypatch):
    import os

    def fails(log):
        raise RuntimeError("no headers")
    with monkeypatch.context() as m:
        m.setattr(ldn_build, "_compile_torch", fails)
        for _ in range(2):
            with pytest.raises(RuntimeError, match="no headers"):
                ldn_build.build()
    assert made == ["libldn.so", "libldn_diag.so"] and os.path.exists(ldn_build.LIB_PATH)
    ldn_build.build()
    assert made == ["libldn.so", "libldn_diag.so", "_ldn_torch.so"]
    ldn_build.build()
    assert len(made) == 3


# ---- the batched references against those that go token by token ----
@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("W,state,bias", [(1, False, False), (4, True, True), (8, True, False), (3, False, True)])
def test_batched_convolution_reference(act, W, state, bias):
    import numpy as np
    from tests import _mixer_ref as ref, _mixer_vec as vec
    r = np.random.default_rng(W)
    B, T, C, lens = 4, 11, 5, [11, 0, 2, 7]
    x, w = r.normal(size=(B, T, C)), r.normal(size=(C, W))
    b, st = r.normal(size=C) if bias else None, r.normal(size=(B, W - 1, C)) if state else None
    dy, dl = r.normal(size=(B, T, C)), r.normal(size=(B, W - 1, C))
    args = (x, w, b, st, lens, act)
    pairs = [(ref.conv(*args), vec.conv(*args)), (ref.conv_bwd(*args, dy, dl), vec.conv_bwd(*args, dy, dl)),
             (ref.conv_bounds(*args, "bf16", dy, dl), vec.conv_bounds(*args, "bf16", dy, dl))]
    inside = (np.arange(T) < np.array(lens)[:, None])[:, :, None]
    for want, got in pairs:
        for a, c in zip(want, got):
            if a.shape == (B, T, C):
                a, c = a * inside, c * inside
            assert np.allclose(a, c, rtol=1e-12, atol=1e-15)


def test_bounds_of_every_state():
    import numpy as np
    from tests import _mixer_ref as ref, _mixer_vec as vec
    r = np.random.default_rng(3)
    B, T, D, G, N, lens = 2, 9, 6, 2, 4, [9, 5]
    p = dict(u=r.normal(size=(B, T, D)), delta=r.normal(size=(B, T, D)), A=-np.abs(r.normal(size=(D, N))),
             B=r.normal(size=(B, T, G, N)), C=r.normal(size=(B, T, G, N)), D=None, z=None, bias=None,
             h0=r.normal(size=(B, D, N)), softplus=True)
    h, e = vec.state_bounds(p, lens)
    assert np.array_equal(h, ref.scan(p, lens)[1])
    assert np.allclose(e[:, -1], ref.scan_bounds(p, lens, "f32")["h"], rtol=1e-12, atol=1e-30)


def test_runs_of_the_convolution_emulated():
    """The launch's run lengths, by the gradient's workspace (it holds a row of sums a block)."""
    from tests import _mixer_vec as vec
    for B, T, C, W in ((1, 1, 1, 1), (4, 2048, 2048, 4), (300, 150, 8, 4), (300, 150, 8, 8), (24, 200, 1100, 4),
                       (3, 3000, 2560, 4), (7, 777, 1028, 3), (2000, 40, 4, 6)):
        cblocks, blocks_sm = -(-C // 128), 4 if W <= 4 else 2
        run = vec.conv_run(B * cblocks, T, W, 4, blocks_sm)
        rblocks = -(-(-(-T // run)) // 4)
        assert ldn.ldn_short_conv_backward_workspace_size(B, T, C, W) == B * rblocks * (W + 1) * C * 4
