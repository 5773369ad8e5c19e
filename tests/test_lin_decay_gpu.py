"""The gradient of linear attention's decays by each token's own measure: every
number within half a step and 2^-16 of the sum of its own terms' absolute values
(`mix_ref`: the same gradient on absolute inputs), however large the gradients of
other tokens of the row are."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_13_amd as gdn
from gated_delta_rule_13_amd import _lib, _mix
from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.gpu_helpers import say
from tests.test_lin_gpu import BF, F32, SCALE, inputs
from tests.test_lin_rounding_gpu import once

pytestmark = pytest.mark.gpu


def reference(a, dO, dS):
    """The exact gradient of log_alpha, and the sums of its terms' absolute values."""
    w = ref.wide(a)
    fn = lambda **k: mix.lin(**k, scale=SCALE)  # noqa: E731
    size = {n: x if n in ("log_alpha", "lens") or x is None else x.abs() for n, x in w.items()}
    absolute = lambda x: None if x is None else x.double().abs()  # noqa: E731
    return [ref.gradients(fn, *args)["log_alpha"] for args in ((w, ["log_alpha"], (dO, dS)),
                                                              (size, ["log_alpha"], (absolute(dO), absolute(dS))))]


def check(a, dO, dS=None):
    want, bound = reference(a, dO, dS)
    got = gdn.gdn_lin_bwd(dO.cuda(), **ref.dev(a), dS_final=None if dS is None else dS.cuda(), scale=SCALE)["dlog_alpha"]
    once("dlog_alpha", got, want, bound)
    return got


def row(dtype, T, dk, dv, seed, strong=0.02, H=2):
    a = inputs(1, H, H, H, T, dk, dv, dtype, seed, "token", False, None, strong)
    return a, ref.rand(ref.gen(seed + 1), 1, H, T, dv, dtype=dtype)


@pytest.mark.parametrize("small", [0.0, 2.0 ** -17])
@pytest.mark.parametrize("dtype,T,dk,dv,start", [(BF, 2100, 64, 64, 1280), (F32, 1000, 40, 64, 512), (BF, 600, 256, 128, 320),
                                                 (BF, 700, 128, 64, 300), (F32, 500, 96, 32, 333)])
def test_documents_of_a_row(dtype, T, dk, dv, start, small):
    """Two documents packed into a row, the first with a gradient of 0 or a small
    one (its own tokens' alone)."""
    say(f"case: lin decays of documents {dtype} T{T} {dk}x{dv} from {start} {small}")
    a, dO = row(dtype, T, dk, dv, T)
    a["log_alpha"][..., start] = -math.inf
    dO[:, :, :start] *= small
    got = check(a, dO)
    assert bool((got[:, :, 1:start].abs().amax(-1) > 0).all()) == (small > 0) and bool((got[:, :, start:].abs() > 0).any())


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 40), (F32, 64, 64), (F32, 256, 32)])
@pytest.mark.parametrize("strong", [0.05, 1.0])
def test_loss_on_the_last_tokens(dtype, dk, dv, strong):
    """A prompt whose own tokens have no loss: what reaches them decays."""
    say(f"case: lin decays of a prompt {dtype} {dk}x{dv} {strong}")
    T = 900
    a, dO = row(dtype, T, dk, dv, dk + dv, strong)
    dO[:, :, :T - 100] = 0
    check(a, dO)


@pytest.mark.parametrize("dtype,T,dk,dv,decay,state,lens", [
    (BF, 700, 128, 128, "token", True, None), (BF, 1100, 40, 64, "resets", True, [1100, 517]), (F32, 500, 72, 40, "token", True, [77, 500]),
    (BF, 300, 200, 256, "token", False, None), (F32, 200, 256, 256, "resets", True, None), (BF, 130, 33, 1, "token", True, [130, 64])])
def test_by_its_own_measure(dtype, T, dk, dv, decay, state, lens):
    say(f"case: lin decays {dtype} T{T} {dk}x{dv} {decay}")
    a = inputs(2, 2, 1, 2, T, dk, dv, dtype, T, decay, state, lens)
    check(a, ref.rand(ref.gen(1), 2, 2, T, dv, dtype=dtype), ref.rand(ref.gen(2), 2, 2, dv, dk) if state else None)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 64, 128), (F32, 40, 32)])
@pytest.mark.parametrize("name,at", [(n, t) for n in ("q", "k", "v", "dO") for t in (0, 30, 75, 127)])
def test_infinities(dtype, dk, dv, name, at):
    """An infinite row written at a token reaches the decays behind it, one read
    there those up to it: the others keep their values, in the token's tile and
    chunk too."""
    T = 200
    a, dO = row(dtype, T, dk, dv, at)
    want, bound = reference(a, dO, None)
    d = {**ref.dev(a), "dO": dO.cuda()}
    d[name] = d[name].clone()
    d[name][0, 1, at, 5] = math.inf
    got = gdn.gdn_lin_bwd(**d, scale=SCALE)["dlog_alpha"]
    keep = slice(0, at + 1) if name in ("k", "v") else slice(at + 1, T)
    once("head without", got[:, 0], want[:, 0], bound[:, 0])
    once("tokens without", got[:, 1, keep], want[:, 1, keep], bound[:, 1, keep])
    rest = got[:, 1, at + 1:] if name in ("k", "v") else got[:, 1, 1:at + 1]
    assert not torch.isfinite(rest).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_decay_for_each_head(dtype):
    """Its gradient sums over tokens and sequences: by the terms' sum too."""
    a = inputs(3, 4, 2, 4, 700, 64, 32, dtype, 3, "head", True, [700, 0, 333])
    check(a, ref.rand(ref.gen(1), 3, 4, 700, 32, dtype=dtype), ref.rand(ref.gen(2), 3, 4, 32, 64))


@pytest.mark.parametrize("dtype,T,dk,dv", [(BF, 37, 64, 128), (BF, 200, 128, 128), (BF, 100, 256, 64), (F32, 150, 64, 64)])
def test_as_exact_as_fp32_arithmetic(dtype, T, dk, dv):
    """In the mean no further from the exact gradient than twice what the
    recurrence in fp32, a token at a time, with its gradient by autograd is."""
    say(f"case: lin decays in fp32 {dtype} T{T} {dk}x{dv}")
    a, dO = row(dtype, T, dk, dv, T, 0.05)
    want, _ = reference(a, dO, None)
    a32 = {n: x.float() if torch.is_tensor(x) and x.is_floating_point() else x for n, x in a.items()}
    la = a32["log_alpha"].clone().requires_grad_(True)
    O, _ = mix.lin(**{**a32, "log_alpha": la}, scale=SCALE)
    plain, = torch.autograd.grad((O * dO.float()).sum(), [la])
    assert plain.dtype is F32
    got = gdn.gdn_lin_bwd(dO.cuda(), **ref.dev(a), scale=SCALE)["dlog_alpha"].cpu()
    off, plain_off = (float((x.double() - want).norm() / want.norm()) for x in (got, plain))
    say(f"off {off:.2e}, fp32 {plain_off:.2e}")
    assert off <= 2 * plain_off


@pytest.mark.parametrize("dtype,T,lens", [(BF, 150, [150, 70, 0]), (BF, 900, [900, 0, 513]), (F32, 700, [1, 700, 320]), (BF, 64, [0, 0, 0])])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 40), (40, 256)])
def test_nothing_of_a_workspace_is_read_before_it_is_written(dtype, T, lens, dk, dv):
    """A workspace full of NaN, with and without segments and empty sequences: the
    same bits as any other."""
    say(f"case: lin bwd on a workspace of NaN {dtype} T{T} {lens} {dk}x{dv}")
    a = ref.dev(inputs(3, 2, 1, 2, T, dk, dv, dtype, T, "token", True, lens))
    dO, dS = ref.rand(ref.gen(1), 3, 2, T, dv, dtype=dtype).cuda(), ref.rand(ref.gen(2), 3, 2, dv, dk).cuda()
    want = gdn.gdn_lin_bwd(dO, **a, dS_final=dS, scale=SCALE)
    assert all(torch.isfinite(x).all() for x in want.values())
    got = {n: torch.full_like(x, math.nan) for n, x in want.items()}
    s = _mix._lin_shape(a["q"], a["k"], a["v"], a["log_alpha"], SCALE, dtype)
    nbytes = gdn.gdn_lin_bwd_workspace_bytes(s)
    ws = torch.full((nbytes,), 0xff, dtype=torch.uint8, device="cuda")
    _lib.check(_lib.load().gdn_lin_bwd(
        ctypes.byref(s), dO.data_ptr(), a["q"].data_ptr(), a["k"].data_ptr(), a["v"].data_ptr(), a["log_alpha"].data_ptr(),
        a["S0"].data_ptr(), dS.data_ptr(), a["lens"].data_ptr(), *(got[n].data_ptr() for n in ("dq", "dk", "dv", "dlog_alpha", "dS0")),
        ws.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream))
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 64, 128), (F32, 40, 64)])
@pytest.mark.parametrize("kind", ["growing", "both ways", "of all sizes"])
def test_decays_of_all_kinds(dtype, dk, dv, kind):
    """States that grow (by e^6 a chunk), that grow and decay, and decays from none
    to all of it beside each other: outputs and every gradient by their own
    terms."""
    say(f"case: lin decays {kind} {dtype} {dk}x{dv}")
    T = 330
    a = inputs(1, 2, 2, 2, T, dk, dv, dtype, 5, "token", True)
    g = ref.gen(6)
    if kind == "growing":
        a["log_alpha"] = 0.1 * torch.rand(1, 2, T, generator=g)
    elif kind == "both ways":
        a["log_alpha"] = 0.5 * torch.randn(1, 2, T, generator=g)
    else:
        pool = torch.tensor([0.0, -1e-4, -0.1, -3.0, -20.0, -60.0, -95.0, -math.inf])
        a["log_alpha"] = pool[torch.randint(0, 8, (1, 2, T), generator=g) * (torch.rand(1, 2, T, generator=g) < 0.3)]
    dO, dS = ref.rand(g, 1, 2, T, dv, dtype=dtype), ref.rand(g, 1, 2, dv, dk)
    w = ref.wide(a)
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    O, S = gdn.gdn_lin_fwd(**ref.dev(a), scale=SCALE)
    once("O", O, wo, bo)
    once("S", S, ws, bs)
    names = ["q", "k", "v", "log_alpha", "S0"]
    size = {n: x if n in ("log_alpha", "lens") or x is None else x.abs() for n, x in w.items()}
    fn = lambda **k: mix.lin(**k, scale=SCALE)  # noqa: E731
    want, bound = ref.gradients(fn, w, names, (dO, dS)), ref.gradients(fn, size, names, (dO.double().abs(), dS.double().abs()))
    got = gdn.gdn_lin_bwd(dO.cuda(), **ref.dev(a), dS_final=dS.cuda(), scale=SCALE)
    for n in names:
        once("d" + n, got["d" + n], want[n], bound[n])
