"""Sizes that the operators around the recurrence refuse, at their exact
boundary, on the CPU: no call here reaches a launch."""
import ctypes

import pytest

from tests.test_abi import lib, lib_nogpu  # noqa: F401
from tests.test_layer_abi import BIG, CALLS, ODD, WORKSPACE, call, conv_shape, norm_shape, ssm_shape

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


def test_gradient_of_many_head_weights(lib_nogpu):  # noqa: F811
    """The sums over w and b of 2^27 numbers each: one thread more than a
    launch counts.  (The forward pass has no such sums.)"""
    query = lib_nogpu.gdn_norm_bwd_workspace_bytes
    for d, fits in ((128, False), (127, True)):
        shape = norm_shape(G=2 ** 20, d=d, w_per_group=1)
        assert (query(ctypes.byref(shape)) < BIG) == fits
        assert call(lib_nogpu, "gdn_norm_bwd", shape, strides=(2 ** 34, 2 ** 27, 128), x=ODD) == 4
        assert ("aligned" in lib_nogpu.gdn_last_error().decode()) == fits
        assert call(lib_nogpu, "gdn_norm_fwd", shape, x=ODD) == 4
        assert "aligned" in lib_nogpu.gdn_last_error().decode()
    # (weights [d]: one sum for all heads)
    assert query(ctypes.byref(norm_shape(G=2 ** 20, d=256))) < BIG


def apart(names):
    """Pointers 16 MiB from each other."""
    return {n: (i + 1) << 24 for i, n in enumerate(names.split())}


@pytest.mark.parametrize("entry", ["gdn_conv_step", "gdn_ssm_step"])
def test_state_in_place_overlaps_nothing(lib_nogpu, entry):  # noqa: F811
    """The state of a token's call, or its output, in the memory of another
    operand: its end, or its beginning."""
    if "conv" in entry:
        shape, state = conv_shape(B=3, T=1, D=64, H=1, x_stride_b=100), "state"
        size = {"x": (2 * 100 + 64) * 2, "weight": 64 * 4 * 4, "bias": 64 * 4, "state": 3 * 3 * 64 * 2, "y": 3 * 64 * 2}
    else:
        strides = {n + "_stride_b": 100 for n in "x dt z b c".split()}
        shape, state = ssm_shape(B=3, T=1, D=64, N=16, G=2, **strides), "h"
        row, bc = (2 * 100 + 64) * 2, (2 * 100 + 32) * 2
        size = {"x": row, "dt": row, "A": 64 * 16 * 4, "Bm": bc, "C": bc, "Dskip": 64 * 4, "z": row, "dt_bias": 64 * 4,
                "h": 3 * 64 * 16 * 4, "y": 3 * 64 * 2}
    names = CALLS[entry][1]
    assert set(size) == set(names.split())
    for out in (state, "y"):
        for other in size:
            if other == out or (out == "y" and other == state):
                continue
            base = apart(names)
            # (4 bytes into the other's end: aligned to either type)
            for moved, to in ((out, base[other] + size[other] - 4), (other, base[out] + size[out] - 4)):
                ptrs = {n: ctypes.c_void_p(v) for n, v in {**base, moved: to}.items()}
                assert call(lib_nogpu, entry, shape, **ptrs) == 4, (out, other, moved)
                assert "overlap" in lib_nogpu.gdn_last_error().decode(), (out, other, moved)
