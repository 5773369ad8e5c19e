"""The short causal convolution on the GPU against the 64-bit reference:
prompts, padded batches, continued states, single tokens, gradients."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, D, W, dtype, seed, state=True, bias=True, lens=None):
    g = ref.gen(seed)
    return {"x": ref.rand(g, B, T, D, dtype=dtype), "weight": ref.rand(g, D, W, std=W ** -0.5),
            "bias": ref.rand(g, D, std=0.2) if bias else None,
            "state0": ref.rand(g, B, W - 1, D, dtype=dtype) if state else None,
            "lens": None if lens is None else torch.tensor(lens, dtype=torch.int32)}


def view_in_wider(x, before, after):
    """x as a slice of a wider row."""
    B, T, D = x.shape
    w = torch.full((B, T, before + D + after), float("nan"), dtype=x.dtype, device=x.device)
    w[:, :, before:before + D] = x
    return w[:, :, before:before + D]


def run(a, **kw):
    B, T, D = a["x"].shape
    H = kw.get("heads") or 1
    W = a["weight"].shape[1]
    y = torch.full((B, T, D) if kw.get("heads") is None else (B, H, T, D // H), float("nan"), dtype=a["x"].dtype,
                   device="cuda")
    st = torch.full((B, W - 1, D), float("nan"), dtype=a["x"].dtype, device="cuda")
    return gdn.gdn_conv_fwd(**ref.dev(a), y=y, state_out=st, **kw)


SHAPES = [  # B, T, D, W, heads, state, bias, act
    (1, 1, 1, 2, None, False, False, None), (2, 1, 8, 4, None, True, True, "silu"), (2, 2, 16, 4, 2, True, True, "silu"),
    (1, 3, 24, 3, 3, False, True, "silu"), (3, 7, 40, 4, None, True, False, "silu"), (2, 8, 33, 2, 3, True, True, None),
    (2, 9, 64, 3, 4, True, True, "silu"), (1, 65, 96, 4, 1, False, True, "silu"), (2, 130, 480, 4, 30, True, True, "silu"),
    (1, 259, 7, 4, 7, True, True, "silu"), (5, 64, 264, 2, None, False, True, "silu"), (1, 1021, 72, 4, 9, True, True, None),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,W,heads,state,bias,act", SHAPES)
def test_forward(dtype, B, T, D, W, heads, state, bias, act):
    say(f"case: conv fwd {dtype} B{B} T{T} D{D} W{W} heads {heads}")
    a = inputs(B, T, D, W, dtype, T + D, state, bias)
    y, st = run(a, heads=heads, act=act)
    want, wst = ref.conv(**ref.wide(a), heads=heads, act=act)
    ref.close("y", y, want)
    assert torch.equal(st.cpu().double(), wst)      # copies, not computed


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("before,after", [(0, 8), (8, 8), (1, 2), (4, 3)])
def test_strided_rows(dtype, before, after):
    """Slices of wider rows, aligned and not: the same bits as dense rows."""
    a = inputs(2, 37, 64, 4, dtype, 3)
    y, st = run(a, heads=4)
    b = dict(a, x=view_in_wider(a["x"], before, after))
    y2, st2 = gdn.gdn_conv_fwd(**ref.dev(b), heads=4)
    assert torch.equal(y, y2) and torch.equal(st, st2)


def test_broadcast_and_transposed_input():
    """A batch stride of 0 (one prompt for all) and rows that are not in order."""
    a = inputs(1, 21, 32, 4, F32, 4, state=False)
    d = ref.dev(a)
    y, _ = gdn.gdn_conv_fwd(d["x"].expand(3, -1, -1), d["weight"], d["bias"])
    one, _ = gdn.gdn_conv_fwd(d["x"], d["weight"], d["bias"])
    assert torch.equal(y, one.expand(3, -1, -1))
    x = ref.rand(ref.gen(5), 21, 3, 32)
    y, _ = gdn.gdn_conv_fwd(x.cuda().transpose(0, 1), d["weight"], d["bias"])
    ref.close("y", y, ref.conv(x.transpose(0, 1).double(), a["weight"].double(), a["bias"].double())[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,lens", [(19, [0, 1, 2, 3, 19, 8]), (70, [70, 69, 64, 65, 0, 5]), (3, [3, 2, 1, 0, -4, 9])])
@pytest.mark.parametrize("state", [False, True])
def test_padded_batch(dtype, T, lens, state):
    """Rows behind a length hold NaN: they reach nothing; outputs there are
    zero; lengths outside [0, T] count as its ends."""
    say(f"case: conv padded {dtype} T{T} lens {lens}")
    a = inputs(6, T, 40, 4, dtype, T, state, True, lens)
    dead = ~ref.live_rows(6, T, a["lens"])
    a["x"][dead] = float("nan")
    y, st = run(a, heads=5)
    want, wst = ref.conv(**ref.wide(a), heads=5)
    ref.close("y", y, want)
    assert torch.equal(st.cpu().double(), wst)
    assert (y.cpu().transpose(1, 2).reshape(6, T, 40)[dead] == 0).all()


def test_in_place_state_and_continuation():
    """A prompt in three calls on one state buffer, and then token by token,
    equals the whole in one call, bit for bit."""
    a = inputs(3, 41, 48, 4, BF, 9)
    d = ref.dev(a)
    whole, wst = gdn.gdn_conv_fwd(d["x"], d["weight"], d["bias"], d["state0"])
    state, parts = d["state0"].clone(), []
    for t0, t1 in ((0, 1), (1, 3), (3, 36)):
        y, out = gdn.gdn_conv_fwd(d["x"][:, t0:t1], d["weight"], d["bias"], state, state_out=state)
        assert out is state
        parts.append(y)
    for t in range(36, 41):
        parts.append(gdn.gdn_conv_step(d["x"][:, t], d["weight"], d["bias"], state)[:, None])
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, wst)


def test_in_place_padded_batch():
    a = inputs(4, 100, 64, 4, BF, 10, True, True, [0, 100, 2, 1])
    d = ref.dev(a)
    _, want = gdn.gdn_conv_fwd(**d)
    state = d["state0"].clone()
    gdn.gdn_conv_fwd(**{**d, "state0": state}, state_out=state)
    assert torch.equal(state, want)


def test_extreme_values():
    """Large and infinite sums through the activation: its limits, no NaN."""
    x = torch.tensor([0.0, 1e-30, -90.0, 90.0, -1e30, 1e30, float("inf"), float("-inf")])[None, :, None].cuda()
    w = torch.tensor([[0.0, 1.0]]).cuda()
    y, _ = gdn.gdn_conv_fwd(x[:, :6], w)
    ref.close("y", y[:, :4], ref.silu(x[:, :4].double().cpu()))
    assert y[0, 4, 0] == 0 and y[0, 5, 0] == 1e30
    # (0 times an infinite row before is NaN by the formula: one row at a time)
    assert gdn.gdn_conv_fwd(x[:, 6:7], w)[0].item() == float("inf")
    assert gdn.gdn_conv_fwd(x[:, 7:8], w)[0].item() == 0


GRADS = [  # B, T, D, W, heads, state, act, lens
    (1, 1, 1, 2, None, False, None, None), (2, 1, 16, 4, None, True, "silu", None), (2, 5, 24, 3, 3, True, "silu", None),
    (1, 61, 40, 4, 5, False, "silu", None), (2, 62, 33, 4, 3, True, "silu", None), (1, 200, 72, 2, None, True, None, None),
    (6, 19, 16, 4, 2, True, "silu", [0, 1, 2, 3, 19, 8]), (3, 130, 264, 4, 33, True, "silu", [130, 61, 2]),
    (2, 9, 7, 3, 1, False, "silu", [4, 9]),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,W,heads,state,act,lens", GRADS)
def test_gradient(dtype, B, T, D, W, heads, state, act, lens):
    say(f"case: conv bwd {dtype} B{B} T{T} D{D} W{W} heads {heads} lens {lens}")
    a = inputs(B, T, D, W, dtype, T * D, state, True, lens)
    g = ref.gen(T)
    dy = ref.rand(g, *((B, T, D) if heads is None else (B, heads, T, D // heads)), dtype=dtype)
    ds = ref.rand(g, B, W - 1, D, dtype=dtype)
    if lens is not None:
        dead = ~ref.live_rows(B, T, a["lens"])
        a["x"][dead] = float("nan")
    got = gdn.gdn_conv_bwd(dy.cuda(), **ref.dev(a), dstate_out=ds.cuda(), act=act)
    fn = lambda **k: ref.conv(**k, heads=heads, act=act)  # noqa: E731
    w = ref.wide(a)
    names = [n for n in ("x", "weight", "bias", "state0") if a[n] is not None]
    want = ref.gradients(fn, w, names, (dy, ds))
    assert set(got) == {"d" + n for n in names}
    for n in names:
        ref.close("d" + n, got["d" + n], want[n])
    again = gdn.gdn_conv_bwd(dy.cuda(), **ref.dev(a), dstate_out=ds.cuda(), act=act)
    assert all(torch.equal(got[k], again[k]) for k in got)      # sums in a fixed order


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,heads", [(262, None), (300, 2), (300, 50), (262, 2), (257, None), (640, 5)])
def test_gradient_pairs_and_slices(dtype, D, heads):
    """Channels that pairs divide, or do not, and slices of wider rows that
    leave the pairs aligned, or not."""
    say(f"case: conv bwd pairs {dtype} D{D} heads {heads}")
    a = inputs(2, 40, D, 4, dtype, D, True, True, [40, 29])
    g = ref.gen(D)
    dy = ref.rand(g, *((2, 40, D) if heads is None else (2, heads, 40, D // heads)), dtype=dtype)
    ds = ref.rand(g, 2, 3, D, dtype=dtype)
    names = ("x", "weight", "bias", "state0")
    want = ref.gradients(lambda **k: ref.conv(**k, heads=heads), ref.wide(a), names, (dy, ds))
    d = ref.dev(a)
    for off in (0, 1, 2):
        rows = torch.full((2, 40, D + 4 + D % 2), float("nan"), dtype=dtype, device="cuda")
        rows[:, :, off:off + D] = d["x"]
        got = gdn.gdn_conv_bwd(dy.cuda(), **{**d, "x": rows[:, :, off:off + D]}, dstate_out=ds.cuda())
        for n in names:
            ref.close("d" + n, got["d" + n], want[n])


def test_gradient_against_differences():
    a = inputs(2, 23, 8, 4, F32, 21)
    g = ref.gen(1)
    dy, ds = ref.rand(g, 2, 23, 8), ref.rand(g, 2, 3, 8)
    got = gdn.gdn_conv_bwd(dy.cuda(), **ref.dev(a), dstate_out=ds.cuda())
    w = ref.wide(a)
    for n in ("x", "weight", "bias", "state0"):
        v = ref.rand(g, *a[n].shape).double()
        want = ref.difference(ref.conv, w, n, v, (dy, ds))
        # each of the gradient's numbers within FP32_TOL of the largest, times
        # the direction; the difference itself within 1e-4^2 of the terms
        mine = got["d" + n].double().cpu()
        slack = (ref.FP32_TOL + 1e-6) * float(mine.abs().max() * v.abs().sum())
        assert abs(float((mine * v).sum()) - want) <= slack, n


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows equal those of a short call."""
    B, T, D = 1, 1_100_000, 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.zeros(B, T, D, dtype=BF, device="cuda")
    x[:, -50:] = torch.randn(B, 50, D, generator=g, device="cuda").to(BF)
    w = torch.randn(D, 4, generator=g, device="cuda")
    y, st = gdn.gdn_conv_fwd(x, w, heads=16)
    want, wst = gdn.gdn_conv_fwd(x[:, -50:], w, heads=16)
    assert torch.equal(y[:, :, -50:], want) and torch.equal(st, wst)
    assert not y[:, :, :-50].any()


def test_refused_calls():
    a = ref.dev(inputs(2, 6, 16, 4, F32, 2))
    bad = [
        (dict(x=a["x"][:, :, ::2]), ValueError), (dict(x=a["x"].half()), TypeError), (dict(x=a["x"][0]), ValueError),
        (dict(weight=a["weight"].to(BF)), TypeError), (dict(weight=a["weight"][:8]), ValueError),
        (dict(weight=torch.zeros(16, 5, device="cuda"), state0=None), gdn.GdnError),
        (dict(weight=torch.zeros(16, 1, device="cuda"), state0=None), gdn.GdnError),
        (dict(state0=a["state0"][:, :2]), ValueError), (dict(state0=a["state0"].to(BF)), TypeError),
        (dict(lens=torch.zeros(2, dtype=torch.int64, device="cuda")), TypeError),
        (dict(lens=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
        (dict(bias=a["bias"].cpu()), ValueError), (dict(heads=3), ValueError), (dict(heads=0), ValueError),
        (dict(act="relu"), ValueError), (dict(x=a["x"].cpu()), ValueError),
        (dict(y=a["x"]), ValueError), (dict(y=torch.zeros(2, 6, 15, device="cuda")), ValueError),
    ]
    for kw, err in bad:
        with pytest.raises(err):
            gdn.gdn_conv_fwd(**{**a, **kw})
    with pytest.raises(ValueError):
        gdn.gdn_conv_step(a["x"][:, 0], a["weight"], a["bias"], None)
    with pytest.raises(ValueError):
        gdn.gdn_conv_bwd(a["x"][:, :5].contiguous(), **a)
