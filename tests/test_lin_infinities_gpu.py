"""Infinite and NaN rows of linear attention reach what is made from them and
nothing else: tokens that come before (in the gradient: after) them, in their own
chunk too, keep the values that they have without, to the rounding of a sum in
another order."""
import math

import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.gpu_helpers import say
from tests.test_lin_gpu import BF, F32, SCALE, inputs

pytestmark = pytest.mark.gpu

# (the place of the bad token: in a chunk of 64 and one of 32, at a chunk's first
# and last token)
PLACES = [(200, 40), (130, 127), (70, 0)]


def agree(name, got, clean, bound):
    """Two sums of the same terms: each off by half a step and 2^-16 of the terms'
    absolute values at most."""
    assert torch.isfinite(got).all(), f"{name}: numbers that are not finite"
    far = (got.double() - clean.double()).abs() - torch.finfo(got.dtype).eps * clean.double().abs() * (1 + 2.0 ** -7)
    assert bool((far.cpu() <= 2.02 * mix.LIN_TOL * bound).all()), (name, float(far.max()))


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("T,at", PLACES)
@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 40), (F32, 64, 64)])
def test_forward(dtype, dk, dv, T, at, name, bad):
    say(f"case: lin fwd {bad} in {name} at {at} of {T} {dtype} {dk}x{dv}")
    a = inputs(1, 2, 2, 2, T, dk, dv, dtype, T + at, "token", True)
    d = ref.dev(a)
    O, _ = gdn.gdn_lin_fwd(**d, scale=SCALE)
    d[name] = d[name].clone()
    d[name][0, 1, at, 3] = bad
    Ob, Sb = gdn.gdn_lin_fwd(**d, scale=SCALE)
    bound = mix.lin_bound(ref.wide(a), scale=SCALE)[0]
    assert torch.equal(Ob[0, 0], O[0, 0])
    agree("O before", Ob[0, 1, :at], O[0, 1, :at], bound[0, 1, :at])
    if name == "q":
        agree("O behind", Ob[0, 1, at + 1:], O[0, 1, at + 1:], bound[0, 1, at + 1:])
        assert torch.isfinite(Sb).all() and not torch.isfinite(Ob[0, 1, at]).any()
    elif name == "v":
        # (one column of the state)
        rest = [c for c in range(dv) if c != 3]
        agree("other columns", Ob[0, 1][:, rest], O[0, 1][:, rest], bound[0, 1][:, rest])
        assert not torch.isfinite(Ob[0, 1, at:, 3]).any() and not torch.isfinite(Sb[0, 1, 3]).any()
    else:
        assert not torch.isfinite(Ob[0, 1, at:]).any() and not torch.isfinite(Sb[0, 1, :, 3]).any()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("name", ["q", "k", "v", "dO"])
@pytest.mark.parametrize("T,at", PLACES)
@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 64), (F32, 64, 64)])
def test_gradient(dtype, dk, dv, T, at, name, bad):
    """dq_t is made of do_t and what was written up to t, dk_t and dv_t of what is
    read from t on and v_t or k_t."""
    say(f"case: lin bwd {bad} in {name} at {at} of {T} {dtype} {dk}x{dv}")
    a = inputs(1, 2, 2, 2, T, dk, dv, dtype, T + at, "token", True)
    dO, dS = ref.rand(ref.gen(1), 1, 2, T, dv, dtype=dtype), ref.rand(ref.gen(2), 1, 2, dv, dk)
    d = {**ref.dev(a), "dO": dO.cuda(), "dS_final": dS.cuda()}
    clean = gdn.gdn_lin_bwd(**d, scale=SCALE)
    d[name] = d[name].clone()
    d[name][0, 1, at, 3] = bad
    got = gdn.gdn_lin_bwd(**d, scale=SCALE)
    w = ref.wide(a)
    size = {n: x if n in ("log_alpha", "lens") or x is None else x.abs() for n, x in w.items()}
    bound = ref.gradients(lambda **k: mix.lin(**k, scale=SCALE), size, ["q", "k", "v"], (dO.double().abs(), dS.double().abs()))
    untouched = {  # of what kind of row: the tokens whose gradient does not hold it
        "q": {"dq": range(T), "dk": range(at + 1, T), "dv": range(at + 1, T)},
        "k": {"dq": range(at), "dk": range(T), "dv": [t for t in range(T) if t != at]},
        "v": {"dq": range(at), "dk": [t for t in range(T) if t != at], "dv": range(T)},
        "dO": {"dq": [t for t in range(T) if t != at], "dk": range(at + 1, T), "dv": range(at + 1, T)}}[name]
    for n, rows in untouched.items():
        rows = list(rows)
        assert torch.equal(got[n][0, 0], clean[n][0, 0])
        if rows:
            agree(n, got[n][0, 1][rows], clean[n][0, 1][rows], bound[n[1:]][0, 1][rows])
