"""Linear attention's outputs in bf16 are rounded once: each within half a step of
its exact value and the error of fp32 outputs, 2^-16 of the sum of its terms'
absolute values (`mix_ref`), with nothing added for roundings of what it is made
from.  Outputs in another type than the rows', too."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.gpu_helpers import say
from tests.test_lin_gpu import BF, F32, SCALE, inputs

pytestmark = pytest.mark.gpu


def once(name, got, want, bound):
    assert tuple(got.shape) == tuple(want.shape), name
    g, w = got.detach().double().cpu(), want.detach().double()
    assert torch.isfinite(g).all(), f"{name}: numbers that are not finite"
    half = torch.finfo(got.dtype).eps / 2
    # (the rounded number may be larger than the exact one by the error)
    off = (g - w).abs() - half * w.abs() - mix.LIN_TOL * bound.detach() * (1 + half)
    worst = float(off.max())
    assert worst <= 1e-30, f"{name}: off by {worst:.3e} more than allowed (largest number {float(w.abs().max()):.3e})"
    if got.dtype is BF and g.numel() >= 4096:
        # One rounding and no more, in the mean: that of numbers off by the terms'
        # error is as large as that of the exact ones to a per cent (the mean square
        # of n uniform errors varies by 0.9 / sqrt(n)).
        rms = lambda x: float((x * x).mean()) ** 0.5  # noqa: E731
        assert rms(g - w) <= 1.05 * rms(w.to(BF).double() - w) + mix.LIN_TOL * rms(bound.detach()), (name, rms(g - w))


CASES = [  # B, H, Hq, Hk, T, dk, dv, decay, state, lens
    (1, 2, 2, 2, 300, 128, 128, "token", True, None), (2, 4, 2, 4, 200, 64, 64, "resets", False, [200, 131]),
    (1, 2, 2, 1, 130, 256, 256, "head", True, None), (1, 1, 1, 1, 700, 96, 32, "none", True, None),
    (1, 2, 1, 2, 140, 72, 40, "token", True, None),
]


@pytest.mark.parametrize("rows,out", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("B,H,Hq,Hk,T,dk,dv,decay,state,lens", CASES)
def test_forward(rows, out, B, H, Hq, Hk, T, dk, dv, decay, state, lens):
    say(f"case: lin fwd once {rows} {out} B{B} H{H}/{Hq}/{Hk} T{T} {dk}x{dv} {decay}")
    a = inputs(B, H, Hq, Hk, T, dk, dv, rows, T + dv, decay, state, lens)
    w = ref.wide(a)
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    O, S = gdn.gdn_lin_fwd(**ref.dev(a), scale=SCALE, o_dtype=out)
    assert O.dtype is out
    once("O", O, wo, bo)
    once("S", S, ws, bs)


@pytest.mark.parametrize("decay", [True, False])
@pytest.mark.parametrize("B,H,Hq,Hk,T,dk,dv,kind,state,lens", CASES)
def test_gradient(decay, B, H, Hq, Hk, T, dk, dv, kind, state, lens):
    """With the decays' gradient and without decays, whose passes differ."""
    say(f"case: lin bwd once B{B} H{H}/{Hq}/{Hk} T{T} {dk}x{dv} {kind} {decay}")
    a = inputs(B, H, Hq, Hk, T, dk, dv, BF, T + dv, kind if decay else "none", state, lens)
    w = ref.wide(a)
    dO, dS = ref.rand(ref.gen(1), B, H, T, dv, dtype=BF), ref.rand(ref.gen(2), B, H, dv, dk)
    names = [n for n in ("q", "k", "v", "S0") if a[n] is not None]
    want = ref.gradients(lambda **k: mix.lin(**k, scale=SCALE), w, names, (dO, dS))
    size = {n: x if n in ("log_alpha", "lens") or x is None else x.abs() for n, x in w.items()}
    bound = ref.gradients(lambda **k: mix.lin(**k, scale=SCALE), size, names, (dO.double().abs(), dS.double().abs()))
    got = gdn.gdn_lin_bwd(dO.cuda(), **ref.dev(a), dS_final=dS.cuda(), scale=SCALE)
    for n in names:
        once("d" + n, got["d" + n], want[n], bound[n])


@pytest.mark.parametrize("rows,out", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("B,H,Hq,Hk,dk,dv", [(2, 4, 2, 4, 64, 64), (1, 3, 3, 1, 45, 33), (3, 2, 2, 2, 256, 200)])
def test_step_in_another_type(rows, out, B, H, Hq, Hk, dk, dv):
    a = inputs(B, H, Hq, Hk, 1, dk, dv, rows, dk + dv)
    w, d = ref.wide(a), ref.dev(a)
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    S = d["S0"].clone()
    tok = [d[n][:, :, 0] for n in ("q", "k", "v", "log_alpha")]
    O = gdn.gdn_lin_step(*tok, S, scale=SCALE, o_dtype=out)
    assert O.dtype is out
    once("O", O, wo[:, :, 0], bo[:, :, 0])
    once("S", S, ws, bs)
    mine = torch.full_like(O, float("nan"))
    S = d["S0"].clone()
    assert gdn.gdn_lin_step(*tok, S, scale=SCALE, O=mine) is mine and torch.equal(mine, O)


@pytest.mark.parametrize("off", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("rows,out", [(BF, BF), (F32, BF), (BF, F32)])
def test_outputs_off_their_places(rows, out, off):
    """O anywhere that its type allows (8 bytes off a 16-byte place, 2 off a 4-byte
    one): the same bits, and nothing around it written."""
    a = ref.dev(inputs(1, 3, 3, 3, 150, 64, 64, rows, 21, "token", True))
    want, _ = gdn.gdn_lin_fwd(**a, scale=SCALE, o_dtype=out)
    n = want.numel()
    buf = torch.full((n + 16,), 7.0, dtype=out, device="cuda")
    got, _ = gdn.gdn_lin_fwd(**a, scale=SCALE, O=buf[off:off + n].view(want.shape))
    assert torch.equal(got, want)
    assert bool((buf[:off] == 7).all()) and bool((buf[off + n:] == 7).all())
