"""The selective state space recurrence on the GPU against the 64-bit
reference: prompts, segments, padded batches, single tokens, gradients."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, D, N, G, dtype, seed, state=True, full=True, lens=None, softplus=True):
    g = ref.gen(seed)
    a = {"x": ref.rand(g, B, T, D, dtype=dtype), "dt": ref.rand(g, B, T, D, dtype=dtype, std=0.5),
         "A": -torch.arange(1, N + 1).float() * torch.exp(ref.rand(g, D, N, std=0.2)),
         "Bm": ref.rand(g, B, T, G, N, dtype=dtype), "C": ref.rand(g, B, T, G, N, dtype=dtype),
         "D": 1 + ref.rand(g, D, std=0.2) if full else None, "z": ref.rand(g, B, T, D, dtype=dtype) if full else None,
         "dt_bias": ref.rand(g, D) - 3 if full else None, "h0": ref.rand(g, B, D, N) if state else None,
         "lens": None if lens is None else torch.tensor(lens, dtype=torch.int32)}
    if not softplus:
        a["dt"] = (a["dt"].float().abs() * 0.1).to(dtype)
        a["dt_bias"] = None
    return a


def run(a, **kw):
    B, T, D = a["x"].shape
    N = a["A"].shape[1]
    y = torch.full((B, T, D), float("nan"), dtype=a["x"].dtype, device="cuda")
    h = torch.full((B, D, N), float("nan"), device="cuda")
    return gdn.gdn_ssm_fwd(**ref.dev(a), y=y, h_final=h, **kw)


def kill(a):
    """NaN behind the lengths, in everything that has rows."""
    dead = ~ref.live_rows(*a["x"].shape[:2], a["lens"])
    for k in ("x", "dt", "Bm", "C", "z"):
        if a[k] is not None:
            a[k][dead] = float("nan")
    return dead


SHAPES = [  # B, T, D, N, G, state, full
    (1, 1, 1, 1, 1, False, False), (2, 1, 64, 16, 1, True, True), (2, 7, 65, 16, 1, True, True),
    (1, 8, 3, 4, 3, True, True), (2, 9, 130, 5, 2, False, True), (1, 31, 200, 8, 1, True, False),
    (3, 64, 24, 24, 2, True, True), (1, 65, 100, 64, 4, True, True), (2, 127, 33, 17, 3, True, True),
    # segments: lengths that end a segment, a token past it, and long
    (1, 128, 64, 16, 1, True, True), (1, 129, 70, 16, 1, False, True), (2, 320, 96, 7, 2, True, True),
    (1, 1000, 48, 16, 1, True, True), (1, 517, 64, 33, 1, True, True), (1, 2048, 16, 1, 1, True, False),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,N,G,state,full", SHAPES)
def test_forward(dtype, B, T, D, N, G, state, full):
    say(f"case: ssm fwd {dtype} B{B} T{T} D{D} N{N} G{G}")
    a = inputs(B, T, D, N, G, dtype, T + D + N, state, full)
    y, h = run(a)
    want, wh = ref.ssm(**ref.wide(a))
    ref.close("y", y, want)
    ref.close("h", h, wh)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_step_sizes_as_they_are(dtype):
    """Without softplus: zeros and a decay rate of zero among them."""
    a = inputs(2, 150, 40, 16, 1, dtype, 4, True, True, softplus=False)
    a["dt"][:, 3:9] = 0
    a["A"][:, 2] = 0
    y, h = run(a, dt_softplus=False)
    want, wh = ref.ssm(**ref.wide(a), dt_softplus=False)
    ref.close("y", y, want)
    ref.close("h", h, wh)


def test_step_sizes_over_their_range():
    """softplus from where it is e^x to where it is x, and decays that leave
    nothing: each number to its own relative accuracy."""
    raw = torch.linspace(-60, 60, 241)[None, None, :].expand(1, 2, -1).contiguous()
    D = raw.shape[2]
    a = {"x": torch.ones(1, 2, D), "dt": raw, "A": torch.zeros(D, 1), "Bm": torch.ones(1, 2, 1, 1),
         "C": torch.ones(1, 2, 1, 1)}
    _, h = gdn.gdn_ssm_fwd(**ref.dev(a))
    want = 2 * torch.logaddexp(raw[0, 0].double(), torch.zeros((), dtype=torch.float64))
    off = ((h[0, :, 0].double().cpu() - want).abs() / want).max()
    # exp2's argument x log2(e) is rounded: 60 * 1.45 * 2^-24 in the exponent,
    # and about 12 roundings more
    assert off <= (60 * 1.45 + 12) * 2.0 ** -24, float(off)
    a = {**a, "A": torch.full((D, 1), -1e4)}
    y, h = gdn.gdn_ssm_fwd(**ref.dev(a))
    assert torch.isfinite(y).all() and torch.isfinite(h).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,lens", [(20, [0, 1, 7, 8, 9, 20]), (300, [300, 0, 64, 65, 200, 5]), (9, [3, -2, 90, 8, 9, 1])])
@pytest.mark.parametrize("state", [False, True])
def test_padded_batch(dtype, T, lens, state):
    say(f"case: ssm padded {dtype} T{T} lens {lens}")
    a = inputs(6, T, 72, 16, 2, dtype, T, state, True, lens)
    dead = kill(a)
    y, h = run(a)
    want, wh = ref.ssm(**ref.wide(a))
    ref.close("y", y, want)
    ref.close("h", h, wh)
    assert (y.cpu()[dead] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,N", [(31, 64), (32, 64), (33, 33), (40, 17), (63, 24)])
def test_short_segments(dtype, T, N):
    """Around the shortest prompts that are cut into segments, padded."""
    say(f"case: ssm short segments {dtype} T{T} N{N}")
    a = inputs(4, T, 70, N, 2, dtype, T + N, True, True, [T, 16, 17, 0])
    dead = kill(a)
    y, h = run(a)
    want, wh = ref.ssm(**ref.wide(a))
    ref.close("y", y, want)
    ref.close("h", h, wh)
    assert (y.cpu()[dead] == 0).all()


@pytest.mark.parametrize("T,n", [(9, 9), (20, 3), (300, 150), (300, 299)])
def test_infinite_last_token(T, n):
    """The infinity of a sequence's last token reaches the final state as one,
    through the empty places of its group and the segments behind it."""
    a = inputs(2, T, 20, 16, 1, F32, T, True, True, [n, n - 1])
    a["x"][0, n - 1] = float("inf")
    a["x"][1, n - 2] = float("-inf")
    y, h = run(a)
    s = torch.nn.functional.softplus(a["dt"].double() + a["dt_bias"].double())
    for b, t in ((0, n - 1), (1, n - 2)):
        want = torch.sign(a["x"][b, t, :, None] * a["Bm"][b, t, 0][None]) * float("inf")
        assert (s[b, t] > 0).all() and torch.equal(h[b].cpu(), want.float())
        assert torch.isfinite(y[b, :t]).all() and not y[b, t + 1:].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_rows(dtype):
    """x, dt, z, B and C as slices of wider rows at odd offsets: the same bits."""
    a = ref.dev(inputs(2, 140, 50, 16, 2, dtype, 8))
    y, h = gdn.gdn_ssm_fwd(**a)
    both = torch.cat([a["x"], a["dt"], a["z"]], 2)
    bc = torch.cat([both[:, :, :3], a["Bm"].flatten(2), a["C"].flatten(2)], 2)
    b = dict(a, x=both[:, :, :50], dt=both[:, :, 50:100], z=both[:, :, 100:],
             Bm=bc[:, :, 3:35].unflatten(2, (2, 16)), C=bc[:, :, 35:].unflatten(2, (2, 16)))
    y2, h2 = gdn.gdn_ssm_fwd(**b)
    assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [40, 400])
def test_in_place_state_and_continuation(dtype, T):
    """A prompt in two calls on one state buffer, then token by token, against
    the reference of the whole."""
    a = inputs(2, T + 6, 70, 16, 1, dtype, T)
    d = ref.dev(a)
    state, parts = d["h0"].clone(), []
    cut = lambda t0, t1: {k: v[:, t0:t1] if k in ("x", "dt", "Bm", "C", "z") else v for k, v in d.items()}  # noqa: E731
    for t0, t1 in ((0, T // 3), (T // 3, T)):
        y, h = gdn.gdn_ssm_fwd(**{**cut(t0, t1), "h0": state}, h_final=state)
        assert h is state
        parts.append(y)
    for t in range(T, T + 6):
        c = {k: v[:, 0] if k in ("x", "dt", "Bm", "C", "z") else v for k, v in cut(t, t + 1).items() if k not in ("h0", "lens")}
        parts.append(gdn.gdn_ssm_step(**c, h=state)[:, None])
    want, wh = ref.ssm(**ref.wide(a))
    ref.close("y", torch.cat(parts, 1), want)
    ref.close("h", state, wh)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,D,N,G,full", [(1, 1, 1, 1, False), (3, 66, 16, 2, True), (5, 30, 7, 3, True), (2, 64, 64, 1, True),
                                          (4, 17, 24, 1, False), (2, 12, 4, 1, True), (65, 200, 8, 1, True)])
def test_step(dtype, B, D, N, G, full):
    say(f"case: ssm step {dtype} B{B} D{D} N{N} G{G}")
    a = inputs(B, 1, D, N, G, dtype, D + N, True, full)
    d = ref.dev(a)
    state = d.pop("h0")
    d.pop("lens")
    y = gdn.gdn_ssm_step(**{k: v[:, 0] if k in ("x", "dt", "Bm", "C", "z") and v is not None else v for k, v in d.items()},
                         h=state)
    want, wh = ref.ssm(**ref.wide(a))
    ref.close("y", y, want[:, 0])
    ref.close("h", state, wh)


def test_strides_of_a_single_row():
    """With one token the stride between tokens is never used: any will do."""
    a = ref.dev(inputs(2, 1, 20, 16, 1, F32, 3))
    y, h = gdn.gdn_ssm_fwd(**a)
    far = a["x"].as_strided((2, 1, 20), (20, 1 << 30, 1))
    y2, h2 = gdn.gdn_ssm_fwd(**{**a, "x": far})
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_step_unaligned_state():
    """A state at an odd address takes the narrow loads."""
    a = inputs(3, 1, 20, 16, 1, F32, 3)
    d = ref.dev(a)
    buf = torch.empty(3 * 20 * 16 + 1, device="cuda")
    h = buf[1:].view(3, 20, 16)
    h.copy_(d["h0"])
    one = {k: d[k][:, 0] for k in ("x", "dt", "Bm", "C", "z")}
    y = gdn.gdn_ssm_step(**one, A=d["A"], D=d["D"], dt_bias=d["dt_bias"], h=h)
    want, wh = ref.ssm(**ref.wide(a))
    ref.close("y", y, want[:, 0])
    ref.close("h", h, wh)


GRADS = [  # B, T, D, N, G, state, full, lens
    (1, 1, 1, 1, 1, False, False, None), (2, 1, 64, 16, 1, True, True, None), (2, 2, 65, 16, 1, True, True, None),
    (1, 8, 12, 4, 3, True, True, None), (2, 9, 70, 5, 2, False, True, None), (1, 31, 40, 8, 1, True, False, None),
    (1, 64, 64, 16, 1, True, True, None), (2, 65, 33, 24, 3, True, True, None), (1, 150, 20, 64, 2, True, True, None),
    (1, 200, 130, 16, 1, True, True, None), (1, 70, 24, 33, 1, True, True, None),
    (6, 20, 72, 16, 2, True, True, [0, 1, 7, 8, 9, 20]), (3, 140, 10, 7, 1, False, True, [140, 64, 65]),
    (2, 70, 16, 40, 1, True, True, [70, 3]),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,N,G,state,full,lens", GRADS)
def test_gradient(dtype, B, T, D, N, G, state, full, lens):
    say(f"case: ssm bwd {dtype} B{B} T{T} D{D} N{N} G{G} lens {lens}")
    a = inputs(B, T, D, N, G, dtype, T * D + N, state, full, lens)
    g = ref.gen(T)
    dy, dh = ref.rand(g, B, T, D, dtype=dtype), ref.rand(g, B, D, N)
    if lens is not None:
        dead = kill(a)
        dy[dead] = float("nan")
    got = gdn.gdn_ssm_bwd(dy.cuda(), **ref.dev(a), dh_final=dh.cuda())
    names = [n for n in ("x", "dt", "A", "Bm", "C", "D", "z", "dt_bias", "h0") if a[n] is not None]
    if lens is not None:
        dy[dead] = 0
    want = ref.gradients(ref.ssm, ref.wide(a), names, (dy, dh))
    assert set(got) == {{"Bm": "dB"}.get(n, "d" + n) for n in names}
    for n in names:
        ref.close("d" + n, got[{"Bm": "dB"}.get(n, "d" + n)], want[n])
    again = gdn.gdn_ssm_bwd(dy.cuda(), **ref.dev(a), dh_final=dh.cuda())
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_gradient_of_step_sizes_as_they_are():
    a = inputs(1, 80, 20, 16, 1, F32, 4, True, True, softplus=False)
    dy = ref.rand(ref.gen(2), 1, 80, 20)
    got = gdn.gdn_ssm_bwd(dy.cuda(), **ref.dev(a), dt_softplus=False)
    want = ref.gradients(lambda **k: ref.ssm(**k, dt_softplus=False), ref.wide(a), ["x", "dt", "A"], (dy, None))
    for n in want:
        ref.close("d" + n, got["d" + n], want[n])


def test_gradient_against_differences():
    a = inputs(1, 75, 6, 16, 2, F32, 21)
    g = ref.gen(1)
    dy, dh = ref.rand(g, 1, 75, 6), ref.rand(g, 1, 6, 16)
    got = gdn.gdn_ssm_bwd(dy.cuda(), **ref.dev(a), dh_final=dh.cuda())
    w = ref.wide(a)
    for n in ("x", "dt", "A", "Bm", "C", "D", "z", "dt_bias", "h0"):
        v = ref.rand(g, *a[n].shape).double()
        want = ref.difference(ref.ssm, w, n, v, (dy, dh), step=1e-5)
        mine = got[{"Bm": "dB"}.get(n, "d" + n)].double().cpu()
        # every number within FP32_TOL of the largest, times the direction, and
        # the difference's own error (step^2 of the third derivative, and
        # 2^-53 / step of the loss) within 1e-6
        slack = (ref.FP32_TOL + 1e-6) * float(mine.abs().max() * v.abs().sum())
        assert abs(float((mine * v).sum()) - want) <= slack, n


def test_offsets_past_32_bits():
    """A state of more than 2^31 numbers, and rows of B and C far apart."""
    B, D, N = 1100, 32768, 64
    assert B * D * N > 2 ** 31
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = torch.zeros(B, D, N, device="cuda")
    h[-1] = torch.randn(D, N, generator=g, device="cuda")
    io = {k: torch.randn(B, D, generator=g, device="cuda").to(BF) for k in ("x", "dt", "z")}
    bc = torch.randn(2, B, 1, N, generator=g, device="cuda").to(BF)
    A = -torch.rand(D, N, generator=g, device="cuda")
    last = h[-1:].clone()
    y = gdn.gdn_ssm_step(io["x"], io["dt"], A, bc[0], bc[1], z=io["z"], h=h)
    y1 = gdn.gdn_ssm_step(io["x"][-1:], io["dt"][-1:], A, bc[0][-1:], bc[1][-1:], z=io["z"][-1:], h=last)
    assert torch.equal(y[-1:], y1) and torch.equal(h[-1:], last)


def test_refused_calls():
    a = ref.dev(inputs(2, 6, 16, 8, 2, F32, 2))
    bad = [
        (dict(x=a["x"][:, :, ::2]), ValueError), (dict(dt=a["dt"].to(BF)), TypeError), (dict(x=a["x"].half()), TypeError),
        (dict(A=a["A"].to(BF)), TypeError), (dict(A=a["A"][:, :4]), ValueError), (dict(A=a["A"].t()), ValueError),
        (dict(Bm=a["Bm"][:, :, :, :4]), ValueError), (dict(Bm=a["Bm"].transpose(2, 3)), ValueError),
        (dict(C=a["C"][:, :5]), ValueError), (dict(z=a["z"][:1]), ValueError), (dict(D=a["D"].cpu()), ValueError),
        (dict(h0=a["h0"].to(BF)), TypeError), (dict(lens=torch.zeros(2, device="cuda")), TypeError),
        (dict(A=torch.zeros(16, 65, device="cuda"), Bm=torch.zeros(2, 6, 2, 65, device="cuda"),
              C=torch.zeros(2, 6, 2, 65, device="cuda"), h0=None), gdn.GdnError),
        (dict(y=a["x"]), ValueError), (dict(x=a["x"].cpu()), ValueError),
        (dict(Bm=torch.zeros(2, 6, 3, 8, device="cuda"), C=torch.zeros(2, 6, 3, 8, device="cuda")), ValueError),
        (dict(h_final=a["h0"].view(-1)[:-1]), ValueError),
    ]
    for kw, err in bad:
        with pytest.raises(err):
            gdn.gdn_ssm_fwd(**{**a, **kw})
    with pytest.raises(ValueError):
        gdn.gdn_ssm_step(a["x"][:, 0], a["dt"][:, 0], a["A"], a["Bm"][:, 0], a["C"][:, 0])
    with pytest.raises(ValueError):
        gdn.gdn_ssm_bwd(a["x"][:, :5].contiguous(), **a)
