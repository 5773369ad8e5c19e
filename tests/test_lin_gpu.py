"""Linear attention with a decay for each head on the GPU, against the 64-bit
reference."""
import ctypes
import math

import pytest
import torch

import gated_delta_rule_13_amd as gdn
from gated_delta_rule_13_amd import _lib, _mix
from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SCALE = 0.3


def inputs(B, H, Hq, Hk, T, dk, dv, dtype, seed, decay="token", state=True, lens=None, strong=0.1):
    g = ref.gen(seed)
    a = {"q": ref.rand(g, B, Hq, T, dk, dtype=dtype), "k": ref.rand(g, B, Hk, T, dk, dtype=dtype),
         "v": ref.rand(g, B, H, T, dv, dtype=dtype), "log_alpha": None, "S0": None, "lens": None}
    if decay == "head":
        a["log_alpha"] = -strong * torch.rand(H, generator=g)
    elif decay != "none":
        la = -strong * torch.rand(B, H, T, generator=g)
        if decay == "resets":
            la[torch.rand(B, H, T, generator=g) < 0.1] = -math.inf
        a["log_alpha"] = la
    if state:
        a["S0"] = ref.rand(g, B, H, dv, dk)
    if lens is not None:
        a["lens"] = torch.tensor(lens, dtype=torch.int32)
    return a


CASES = [  # B, H, Hq, Hk, T, dk, dv, decay, state, lens
    (1, 1, 1, 1, 1, 1, 1, "token", True, None), (1, 2, 2, 2, 3, 8, 5, "token", False, None),
    (2, 2, 1, 2, 17, 16, 16, "none", True, None), (2, 3, 3, 1, 64, 32, 32, "head", True, None),
    (1, 2, 2, 2, 65, 64, 64, "token", True, None), (2, 4, 2, 4, 127, 128, 128, "token", True, [127, 64]),
    (3, 2, 2, 2, 130, 96, 192, "token", False, [130, 0, 65]), (1, 1, 1, 1, 200, 256, 256, "token", True, None),
    (2, 6, 2, 3, 100, 72, 40, "resets", True, [100, 33]), (1, 2, 1, 1, 150, 33, 100, "resets", False, None),
    (1, 2, 2, 2, 129, 130, 20, "head", True, [1]), (1, 1, 1, 1, 300, 40, 256, "none", False, [299]),
    (1, 3, 3, 3, 31, 256, 8, "token", True, None), (2, 1, 1, 1, 96, 100, 129, "token", True, [5, 96]),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hq,Hk,T,dk,dv,decay,state,lens", CASES)
def test_forward(dtype, B, H, Hq, Hk, T, dk, dv, decay, state, lens):
    say(f"case: lin fwd {dtype} B{B} H{H}/{Hq}/{Hk} T{T} {dk}x{dv} {decay}")
    a = inputs(B, H, Hq, Hk, T, dk, dv, dtype, T + dk, decay, state, lens)
    O = torch.full((B, H, T, dv), float("nan"), dtype=dtype, device="cuda")
    S = torch.full((B, H, dv, dk), float("nan"), device="cuda")
    gdn.gdn_lin_fwd(**ref.dev(a), scale=SCALE, O=O, S_final=S)
    w = ref.wide(a)
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    mix.within("O", O, wo, bo)
    mix.within("S", S, ws, bs)
    if dtype is BF:
        mix.within("O in fp32", gdn.gdn_lin_fwd(**ref.dev(a), scale=SCALE, o_dtype=F32)[0], wo, bo)


def check_gradient(a, dO, dS, got, scale=SCALE):
    w = ref.wide(a)
    names = [n for n in ("q", "k", "v", "log_alpha", "S0") if a[n] is not None]
    want = ref.gradients(lambda **k: mix.lin(**k, scale=scale), w, names, (dO, dS))
    absolute = {n: x if n in ("log_alpha", "lens") or x is None else x.abs() for n, x in w.items()}
    bound = ref.gradients(lambda **k: mix.lin(**k, scale=scale), absolute, names,
                          (dO.double().abs(), None if dS is None else dS.double().abs()))
    assert set(got) == {"d" + n for n in names}
    for n in names:
        b = bound[n]
        if n == "log_alpha":
            B, H, T, _ = a["v"].shape
            parts = (absolute["q"] * bound["q"]).sum(-1).max() + (absolute["k"] * bound["k"]).sum(-1).max()
            b = b + math.sqrt(T) * parts * (math.sqrt(B * T) if b.dim() == 1 else 1)
        mix.within("d" + n, got["d" + n], want[n], b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hq,Hk,T,dk,dv,decay,state,lens", CASES)
def test_gradient(dtype, B, H, Hq, Hk, T, dk, dv, decay, state, lens):
    say(f"case: lin bwd {dtype} B{B} H{H}/{Hq}/{Hk} T{T} {dk}x{dv} {decay}")
    a = inputs(B, H, Hq, Hk, T, dk, dv, dtype, T + dk, decay, state, lens)
    g = ref.gen(9)
    dO, dS = ref.rand(g, B, H, T, dv, dtype=dtype), ref.rand(g, B, H, dv, dk) if state else None
    d = ref.dev(a)
    call = lambda: gdn.gdn_lin_bwd(dO.cuda(), **d, dS_final=None if dS is None else dS.cuda(), scale=SCALE)  # noqa: E731
    got = call()
    check_gradient(a, dO, dS, got)
    again = call()
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,decay", [(1100, "token"), (900, "resets"), (1029, "head"), (700, "none")])
def test_segments(dtype, T, decay):
    """Few heads on long sequences: segments that run at once."""
    say(f"case: lin segments {dtype} T{T} {decay}")
    a = inputs(2, 2, 1, 2, T, 40, 64, dtype, T, decay, True, [T, 517], strong=0.02)
    w = ref.wide(a)
    O, S = gdn.gdn_lin_fwd(**ref.dev(a), scale=SCALE)
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    mix.within("O", O, wo, bo)
    mix.within("S", S, ws, bs)
    dO, dS = ref.rand(ref.gen(1), 2, 2, T, 64, dtype=dtype), ref.rand(ref.gen(2), 2, 2, 64, 40)
    check_gradient(a, dO, dS, gdn.gdn_lin_bwd(dO.cuda(), **ref.dev(a), dS_final=dS.cuda(), scale=SCALE))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv,lens", [(32, 32, None), (64, 64, [400, 321]), (96, 96, [399, 256]), (128, 128, None), (256, 256, [385, 400]),
                                        (128, 64, [193, 400]), (64, 256, None), (256, 96, None), (104, 40, None), (16, 128, None)])
def test_many_chunks(dtype, dk, dv, lens):
    """More chunks than LDS holds at once, in every built size of rows."""
    say(f"case: lin chunks {dtype} {dk}x{dv}")
    T = 400
    a = inputs(2, 2, 2, 2, T, dk, dv, dtype, dk + dv, "token", True, lens)
    w = ref.wide(a)
    O, S = gdn.gdn_lin_fwd(**ref.dev(a), scale=SCALE)
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    mix.within("O", O, wo, bo)
    mix.within("S", S, ws, bs)
    dO, dS = ref.rand(ref.gen(1), 2, 2, T, dv, dtype=dtype), ref.rand(ref.gen(2), 2, 2, dv, dk)
    check_gradient(a, dO, dS, gdn.gdn_lin_bwd(dO.cuda(), **ref.dev(a), dS_final=dS.cuda(), scale=SCALE))


@pytest.mark.parametrize("strong", [1.0, 8.0, 60.0])
def test_strong_decays(strong):
    """Chunks whose decay spans up to e^-3000: no factor leaves its range, and
    the decay's gradient keeps its own scale."""
    a = inputs(1, 2, 2, 2, 150, 64, 64, BF, 5, "token", True, None, strong)
    w = ref.wide(a)
    O, S = gdn.gdn_lin_fwd(**ref.dev(a), scale=SCALE)
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    mix.within("O", O, wo, bo)
    mix.within("S", S, ws, bs)
    dO = ref.rand(ref.gen(1), 1, 2, 150, 64, dtype=BF)
    got = gdn.gdn_lin_bwd(dO.cuda(), **ref.dev(a), scale=SCALE)
    check_gradient(a, dO, None, got)
    want = ref.gradients(lambda **k: mix.lin(**k, scale=SCALE), w, ["log_alpha"], (dO, None))["log_alpha"]
    # (strong decays leave pairs of neighbours, nothing to cancel)
    err = float((got["dlog_alpha"].double().cpu() - want).abs().max() / want.abs().max())
    assert err < 1e-4, err


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hq,Hk,dk,dv,decay", [
    (1, 1, 1, 1, 1, 1, "token"), (3, 4, 2, 1, 16, 7, "token"), (2, 2, 2, 2, 64, 64, "none"), (5, 6, 3, 2, 128, 128, "head"),
    (1, 30, 30, 30, 96, 192, "token"), (2, 2, 1, 2, 256, 256, "resets"), (2, 3, 3, 3, 45, 33, "token"), (1, 2, 2, 2, 200, 130, "token")])
def test_step(dtype, B, H, Hq, Hk, dk, dv, decay):
    """Tokens one by one, after a prompt: as the reference on the whole."""
    say(f"case: lin step {dtype} B{B} H{H}/{Hq}/{Hk} {dk}x{dv} {decay}")
    T, new = 20, 3
    a = inputs(B, H, Hq, Hk, T + new, dk, dv, dtype, dk + dv, decay)
    w = ref.wide(a)
    d = ref.dev(a)
    tok = lambda x, t: None if x is None else x if x.dim() == 1 else x[:, :, t]  # noqa: E731
    first = {n: x if n in ("S0", "lens") or x is None or x.dim() == 1 else x[:, :, :T] for n, x in d.items()}
    _, S = gdn.gdn_lin_fwd(**first, scale=SCALE)
    out = [gdn.gdn_lin_step(d["q"][:, :, t], d["k"][:, :, t], d["v"][:, :, t], tok(d["log_alpha"], t), S, scale=SCALE)
           for t in range(T, T + new)]
    (wo, ws), (bo, bs) = mix.lin(**w, scale=SCALE), mix.lin_bound(w, scale=SCALE)
    mix.within("O", torch.stack(out, 2), wo[:, :, T:], bo[:, :, T:])
    mix.within("S", S, ws, bs)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_views(dtype):
    """Slices of a projection, rows off their 16-byte places, a broadcast
    batch, decays [B, T, H], the state in place: as dense copies, to the bit."""
    B, H, T, dk, dv = 2, 3, 90, 40, 24
    g = ref.gen(4)
    proj = ref.rand(g, B, T, H * (2 * dk + dv) + 3, dtype=dtype).cuda()
    la = -0.1 * torch.rand(B, T, H, generator=g).cuda()
    for first in (0, 1):
        q = proj[:, :, first:first + H * dk].unflatten(2, (H, dk)).transpose(1, 2)
        k = proj[:1, :, first + H * dk:first + 2 * H * dk].unflatten(2, (H, dk)).transpose(1, 2).expand(B, H, T, dk)
        v = proj[:, :, first + 2 * H * dk:first + H * (2 * dk + dv)].unflatten(2, (H, dv)).transpose(1, 2)
        S0 = ref.rand(g, B, H, dv, dk).cuda()
        views, dense = (q, k, v, la.transpose(1, 2)), tuple(x.contiguous() for x in (q, k, v, la.transpose(1, 2)))
        O, S = gdn.gdn_lin_fwd(*dense, S0)
        S1 = S0.clone()
        O1, _ = gdn.gdn_lin_fwd(*views, S1, S_final=S1)
        assert torch.equal(O, O1) and torch.equal(S, S1)
        dO = ref.rand(g, B, H, T, dv, dtype=dtype).cuda()
        x, y = gdn.gdn_lin_bwd(dO, *views, S0), gdn.gdn_lin_bwd(dO, *dense, S0)
        assert all(torch.equal(x[n], y[n]) for n in x)
        one = lambda t: [x[:, :, 5] for x in t]  # noqa: E731
        S1, S2 = S0.clone(), S0.clone()
        O1, O2 = gdn.gdn_lin_step(*one(views), S1), gdn.gdn_lin_step(*one(dense), S2)
        assert torch.equal(S1, S2)
        # (rows off their places: the sum over d_k in another order, each of 40
        # additions off by 2^-24 of the terms so far at most, and a rounding each)
        terms = S1.double().abs() @ q[:, :, 5].double().abs()[..., None]
        far = (O1.double() - O2.double()).abs() - torch.finfo(dtype).eps * O2.double().abs()
        assert bool((far <= 2 * dk * 2.0 ** -24 * terms[..., 0] * 1.01).all())


def test_padding_and_other_sequences():
    """NaN behind a sequence's end reaches nothing; NaN and infinity in one
    sequence reach that sequence and head only."""
    a = inputs(3, 2, 2, 2, 100, 64, 48, BF, 7, lens=[100, 40, 0])
    clean = ref.dev(a)
    bad = {n: x.clone() if torch.is_tensor(x) else x for n, x in clean.items()}
    for n in ("q", "k", "v"):
        bad[n][1, :, 40:] = float("nan")
        bad[n][2] = float("inf")
    bad["log_alpha"][1, :, 40:] = float("nan")
    dO = ref.rand(ref.gen(3), 3, 2, 100, 48, dtype=BF).cuda()
    dbad = dO.clone()
    dbad[1, :, 40:] = float("nan")
    for x, y in zip(gdn.gdn_lin_fwd(**clean), gdn.gdn_lin_fwd(**bad)):
        assert torch.equal(x, y)
    x, y = gdn.gdn_lin_bwd(dO, **clean), gdn.gdn_lin_bwd(dbad, **bad)
    assert all(torch.equal(x[n], y[n]) for n in x)
    assert all(not x[n][1, :, 40:].any() and not x[n][2].any() for n in ("dq", "dk", "dv", "dlog_alpha"))
    bad = {n: v.clone() if torch.is_tensor(v) else v for n, v in clean.items()}
    bad["k"][0, 1, 30] = float("nan")
    bad["v"][1, 0, 3] = float("inf")
    O, _ = gdn.gdn_lin_fwd(**bad)
    ok, _ = gdn.gdn_lin_fwd(**clean)
    assert torch.equal(O[0, 0], ok[0, 0]) and torch.equal(O[1, 1], ok[1, 1]) and not torch.isfinite(O[0, 1].float()).all()


def test_agrees_with_the_delta_rule_without_erasing():
    """gdn_chunk_fwd_eta with erase strength 0 and write strength 1 is the same
    recurrence (its operands are fp16: 2e-3 of the largest)."""
    a = ref.dev(inputs(2, 2, 2, 2, 200, 64, 64, BF, 8))
    one = torch.ones(2, 2, 200, device="cuda")
    unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).to(BF)  # noqa: E731
    q, k = unit(a["q"]), unit(a["k"])
    O, S = gdn.gdn_chunk_fwd_eta(q, k, a["v"], a["log_alpha"].exp(), 0 * one, one, a["S0"])
    O1, S1 = gdn.gdn_lin_fwd(q, k, a["v"], a["log_alpha"], a["S0"], o_dtype=F32)
    for x, y in ((O, O1), (S, S1)):
        assert float((x - y).abs().max() / y.abs().max()) < 2e-3


@pytest.mark.parametrize("name", ["q", "k", "v", "log_alpha", "S0"])
def test_gradient_against_differences(name):
    """The kernel's gradient along a direction against central differences of
    the kernel's own forward pass in fp32: step^2 of the third derivative and
    2^-16 of the loss's terms over the step."""
    a = inputs(1, 2, 1, 2, 70, 24, 16, F32, 11)
    g = ref.gen(12)
    dO, dS = ref.rand(g, 1, 2, 70, 16).cuda(), ref.rand(g, 1, 2, 16, 24).cuda()
    d = ref.dev(a)
    step = 2.0 ** -5
    way = ref.rand(g, *a[name].shape, std=0.1).cuda()

    def loss(s):
        O, S = gdn.gdn_lin_fwd(**{**d, name: d[name] + s * way}, scale=SCALE)
        return float((O.double() * dO).sum() + (S.double() * dS).sum())
    got = gdn.gdn_lin_bwd(dO, **d, dS_final=dS, scale=SCALE)
    slope = float((got["d" + name].double() * way).sum())
    want = (loss(step) - loss(-step)) / (2 * step)
    w = {n: x if n in ("log_alpha", "lens") or x is None else x.abs() for n, x in ref.wide(a).items()}
    size = sum(float((x.abs() ** 2 * y.cpu().double() ** 2).sum()) ** 0.5 for x, y in zip(mix.lin(**w, scale=SCALE), (dO, dS)))
    # (q, k, v and S0 enter linearly; log_alpha's third derivative is at most the
    # tokens it acts over, cubed, times the direction's cube)
    assert abs(slope - want) < 2.0 ** -16 * size / step + (2e-2 * abs(want) + 0.05 if name == "log_alpha" else 1e-4 * abs(want)), (slope, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay,T", [("token", 200), ("head", 200), ("token", 700)])
def test_gradient_without_the_decays(dtype, decay, T):
    """The C entry without dlog_alpha and dS0: what is left is held to the same
    bounds (in one pass, and in segments)."""
    say(f"case: lin bwd without dlog_alpha {dtype} {decay} T{T}")
    a = inputs(2, 2, 1, 2, T, 40, 64, dtype, T, decay, True, [T, T - 61])
    dO, dS = ref.rand(ref.gen(1), 2, 2, T, 64, dtype=dtype), ref.rand(ref.gen(2), 2, 2, 64, 40)
    d, do, ds = ref.dev(a), dO.cuda(), dS.cuda()
    full = gdn.gdn_lin_bwd(do, **d, dS_final=ds, scale=SCALE)
    some = {n: torch.full_like(full[n], math.nan) for n in ("dq", "dk", "dv")}
    s = _mix._lin_shape(d["q"], d["k"], d["v"], d["log_alpha"], SCALE, dtype)
    nbytes = gdn.gdn_lin_bwd_workspace_bytes(s)
    ws = torch.full((nbytes,), 0xff, dtype=torch.uint8, device="cuda")
    _lib.check(_lib.load().gdn_lin_bwd(
        ctypes.byref(s), do.data_ptr(), d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), d["log_alpha"].data_ptr(),
        d["S0"].data_ptr(), ds.data_ptr(), d["lens"].data_ptr(), some["dq"].data_ptr(), some["dk"].data_ptr(),
        some["dv"].data_ptr(), None, None, ws.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream))
    check_gradient(a, dO, dS, {**full, **some})
