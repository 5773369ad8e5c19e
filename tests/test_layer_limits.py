"""Sizes that the operators around the recurrence refuse, at their exact
boundary, on the CPU: no call here reaches a launch."""
import ctypes

import pytest

from tests.test_abi import lib, lib_nogpu  # noqa: F401
from tests.test_layer_abi import BIG, CALLS, ODD, WORKSPACE, call

MOST = 2 ** 31 - 128                # tokens: the kernels walk them, a tile ahead, in 32 bits


@pytest.mark.parametrize("entry", ["gdn_conv_fwd", "gdn_conv_bwd", "gdn_ssm_fwd"])
@pytest.mark.parametrize("past", [1, 64, 127])
def test_tokens(lib_nogpu, entry, past):  # noqa: F811
    """(The scan's gradient has more threads than a launch counts before that.)"""
    one = dict(B=1, D=1, H=1) if "conv" in entry else dict(B=1, D=1, G=1, N=1)
    shape = CALLS[entry][0]
    assert call(lib_nogpu, entry, shape(T=MOST, **one), x=ODD) == 4
    assert "aligned" in lib_nogpu.gdn_last_error().decode()          # (accepted: refused for its pointer)
    assert call(lib_nogpu, entry, shape(T=MOST + past, **one), x=ODD) == 4
    assert "T must be at most" in lib_nogpu.gdn_last_error().decode()
    if entry in WORKSPACE:
        query = getattr(lib_nogpu, entry + "_workspace_bytes")
        assert query(ctypes.byref(shape(T=MOST, **one))) < BIG
        assert query(ctypes.byref(shape(T=MOST + past, **one))) == BIG
