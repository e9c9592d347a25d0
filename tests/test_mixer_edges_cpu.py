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
