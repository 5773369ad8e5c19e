"""Outputs passed in that lie in the memory of another operand are refused,
whichever operand it is."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn

pytestmark = pytest.mark.gpu

B, T, D, N = 2, 5, 12, 4
ROWS = {"x": (B, T, D), "dt": (B, T, D), "z": (B, T, D), "Bm": (B, T, 1, N), "C": (B, T, 1, N)}
CONV = {"x": (B, T, D), "weight": (D, 4), "bias": (D,), "state0": (B, 3, D), "lens": (B,)}
SSM = {**ROWS, "A": (D, N), "D": (D,), "dt_bias": (D,), "h0": (B, D, N), "lens": (B,)}
NORM = {"x": (B, T, 3, 4), "weight": (3, 4), "bias": (3, 4), "z": (B, T, 3, 4)}


def one(shapes):
    """The shapes of one token's operands."""
    return {k: (s[0],) + s[2:] if k in ("x", "dt", "z", "Bm", "C") else s for k, s in shapes.items() if k != "lens"}


def step_shapes(shapes, state, name):
    out = one(shapes)
    out[name] = out.pop(state)
    return out


ENTRIES = {  # entry: operands, outputs and their shapes
    "gdn_conv_fwd": (CONV, {"y": (B, T, D), "state_out": (B, 3, D)}),
    "gdn_conv_step": (step_shapes(CONV, "state0", "state"), {"y": (B, D)}),
    "gdn_ssm_fwd": (SSM, {"y": (B, T, D), "h_final": (B, D, N)}),
    "gdn_ssm_step": (step_shapes(SSM, "h0", "h"), {"y": (B, D)}),
    "gdn_norm_fwd": (NORM, {"y": (B, T, 3, 4)}),
}
IN_PLACE = {("gdn_conv_step", "state"), ("gdn_ssm_step", "h")}
CASES = [(e, out, other) for e, (ins, outs) in ENTRIES.items() for out in outs for other in list(ins) + list(outs) if other != out]
CASES += [(e, state, other) for e, state in sorted(IN_PLACE) for other in ENTRIES[e][0] if other != state]


def tensor(name, shape, memory=None):
    n = 1
    for s in shape:
        n *= s
    flat = torch.zeros(n, device="cuda") if memory is None else memory[:n]
    return (flat.view(torch.int32) if name == "lens" else flat).view(shape)


@pytest.mark.parametrize("entry,out,other", CASES)
def test_overlap(entry, out, other):
    ins, outs = ENTRIES[entry]
    shapes = {**ins, **outs}
    args = {k: tensor(k, s) for k, s in ins.items()}
    getattr(gdn, entry)(**args, **{k: tensor(k, s) for k, s in outs.items()})       # (apart: fine)
    memory = torch.zeros(4096, device="cuda")
    count = args[other].numel() if other in args else tensor(other, outs[other]).numel()
    args[other] = tensor(other, shapes[other], memory)
    args[out] = tensor(out, shapes[out], memory[count - 1:])
    with pytest.raises((ValueError, gdn.GdnError), match="overlap"):
        getattr(gdn, entry)(**args)
