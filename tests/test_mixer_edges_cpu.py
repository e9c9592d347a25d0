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
