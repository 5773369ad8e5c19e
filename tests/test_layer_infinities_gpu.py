"""Infinite numbers in the operators around the recurrence: an output is what
the formula gives, wherever the infinity falls in a kernel's groups, tiles and
padding.  Inputs are positive where the formula would otherwise subtract two
infinities; what the formula leaves undefined is not compared."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def meets(name, got, want):
    """got where the fp64 reference has a value: infinities alike, the finite
    numbers as layer_ref.close takes them (the largest of the finite ones)."""
    assert tuple(got.shape) == tuple(want.shape), (name, tuple(got.shape), tuple(want.shape))
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    wild = torch.isinf(w)
    bad = wild & (g != w)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {int(wild.sum())} infinities are not, e.g. {g[bad][:3].tolist()}"
    calm = torch.isfinite(w)
    if calm.any():
        ref.close(name, got.detach().cpu()[calm], w[calm])


def inputs(T, D, N, dtype, seed, D_=True, z=True):
    """(Decay rates up to about 3: the decay over a segment of tokens stays a
    number of fp32 above 0, whose product with an infinity is one.)"""
    g = ref.gen(seed)
    pos = lambda *s, **k: ref.rand(g, *s, **k).abs() + 0.01  # noqa: E731
    return {"x": pos(1, T, D).to(dtype), "dt": ref.rand(g, 1, T, D, std=0.5, dtype=dtype),
            "A": -2 * torch.arange(1, N + 1).float() / N * torch.exp(ref.rand(g, D, N, std=0.2)),
            "Bm": pos(1, T, 1, N).to(dtype), "C": pos(1, T, 1, N).to(dtype), "D": pos(D) if D_ else None,
            "z": pos(1, T, D).to(dtype) if z else None, "dt_bias": ref.rand(g, D) - 3, "h0": pos(1, D, N)}


ROWS = ("x", "dt", "Bm", "C", "z")


def padded(a, T, names=ROWS):
    """The sequence in a batch padded to T rows, NaN behind it."""
    n = a["x"].shape[1]
    out = dict(a, lens=torch.tensor([n], dtype=torch.int32))
    for k in names:
        if a.get(k) is not None:
            out[k] = torch.full((1, T) + tuple(a[k].shape[2:]), float("nan"), dtype=a[k].dtype)
            out[k][:, :n] = a[k]
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 3, 5, 7, 12, 17, 24, 33, 48, 4, 16, 64])
@pytest.mark.parametrize("T", [1, 13, 200])
@pytest.mark.parametrize("where", ["x", "dt"])
def test_scan_states(dtype, N, T, where):
    """Any number of states: those that fill up a kernel's size take no part."""
    say(f"case: infinite {where} {dtype} T{T} N{N}")
    a = inputs(T, 20, N, dtype, T + N)
    a[where][0, T // 2, 3] = INF
    want, wh = ref.ssm(**ref.wide(a))
    assert torch.isinf(want).any() and torch.isfinite(want).any()
    y, h = gdn.gdn_ssm_fwd(**ref.dev(a))
    meets("y", y, want)
    meets("h", h, wh)
    if T == 1:
        d = {k: v[:, 0] if k in ROWS else v for k, v in ref.dev(a).items()}
        state = d.pop("h0")
        meets("y", gdn.gdn_ssm_step(**d, h=state), want[:, 0])
        meets("h", state, wh)


def gradient(a, dy, dh, **kw):
    got = gdn.gdn_ssm_bwd(dy.cuda(), **ref.dev(a), dh_final=dh.cuda(), **kw)
    return {("B" if k == "dB" else k): v for k, v in got.items()}


def check_gradient(a, dy, dh, T=None):
    """Against autograd through the formula, the sequence alone or padded to T
    rows."""
    n = a["x"].shape[1]
    names = [k for k in ("x", "dt", "A", "Bm", "C", "D", "z", "dt_bias", "h0") if a[k] is not None]
    want = ref.gradients(ref.ssm, ref.wide(a), names, (dy, dh))
    if T is not None:
        rows = padded(dict(a, dy=dy), T, ROWS + ("dy",))
        dy = rows.pop("dy")
        a = rows
    got = gradient(a, dy, dh)
    for k in names:
        v = got["B" if k == "Bm" else "d" + k]
        if k in ROWS and T is not None:
            assert not v[:, n:].any(), k
            v = v[:, :n]
        meets("d" + k, v, want[k])
    return want


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 3, 5, 7, 12, 24, 33, 48, 4, 16, 64])
@pytest.mark.parametrize("where", ["x", "dy", "dt"])
@pytest.mark.parametrize("T,t", [(24, 9), (88, 49)])
def test_scan_gradient_states(dtype, N, where, T, t):
    say(f"case: infinite {where}, gradient {dtype} N{N} T{T}")
    a = inputs(T, 64, N, dtype, N)
    g = ref.gen(N)
    dy, dh = ref.rand(g, 1, T, 64).abs().to(dtype), ref.rand(g, 1, 64, N).abs()
    (dy if where == "dy" else a[where])[0, t, 3] = INF
    want = check_gradient(a, dy, dh)
    assert any(torch.isinf(v).any() for v in want.values())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [11, 90])
def test_scan_without_skip(dtype, T):
    """No skip term: not 0 times an infinite x."""
    a = inputs(T, 24, 16, dtype, T, D_=False, z=False)
    a["x"][0, 6, 5] = INF
    want, _ = ref.ssm(**ref.wide(a))
    y, _ = gdn.gdn_ssm_fwd(**ref.dev(a))
    assert torch.isinf(want).any()
    meets("y", y, want)
    one = {k: v[:, 6] if k in ROWS else v for k, v in ref.dev({k: v for k, v in a.items() if v is not None}).items()}
    state = one.pop("h0")
    first, _ = ref.ssm(**{k: v[:, 6:7] if k in ROWS and v is not None else v for k, v in ref.wide(a).items()})
    meets("y", gdn.gdn_ssm_step(**one, h=state), first[:, 0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("where", ["x", "dy"])
def test_scan_gradient_without_skip(dtype, where):
    a = inputs(16, 64, 16, dtype, 4, D_=False)
    g = ref.gen(5)
    dy, dh = ref.rand(g, 1, 16, 64).abs().to(dtype), ref.rand(g, 1, 64, 16).abs()
    (dy if where == "dy" else a["x"])[0, 9, 3] = INF
    check_gradient(a, dy, dh)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 15, 16, 17, 70])
@pytest.mark.parametrize("where", ["x", "Bm", "C"])
def test_scan_gradient_of_the_last_token(dtype, n, where):
    """The infinity of a sequence's last token, wherever its length falls in a
    group of tokens: as the sequence alone, with no rows behind it."""
    say(f"case: infinite last {where}, gradient {dtype} n{n}")
    a = inputs(n, 64, 16, dtype, n)
    g = ref.gen(n)
    dy, dh = ref.rand(g, 1, n, 64).abs().to(dtype), ref.rand(g, 1, 64, 16).abs()
    a[where][0, n - 1, 0 if where != "x" else 3] = INF
    check_gradient(a, dy, dh)
    check_gradient(a, dy, dh, T=n + 13)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [20, 70])
@pytest.mark.parametrize("n", [8, 40])
@pytest.mark.parametrize("where", ["x", "dy", "dt"])
def test_scan_gradient_of_the_last_channel(dtype, D, n, where):
    """Lanes without a channel add nothing to the sums over channels, also
    where the channel beside them is infinite."""
    a = inputs(n, D, 16, dtype, n)
    g = ref.gen(n)
    dy, dh = ref.rand(g, 1, n, D).abs().to(dtype), ref.rand(g, 1, D, 16).abs()
    (dy if where == "dy" else a[where])[0, 5, D - 1] = INF
    check_gradient(a, dy, dh)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 4, 7, 20])
def test_convolution_gradient(dtype, W, T):
    """An infinite row at every place: rows of other tiles, and those that
    stand behind a sequence's end, add nothing to the taps' gradients."""
    g = ref.gen(T + W)
    x, w, b = ref.rand(g, 1, T, 6, dtype=dtype), ref.rand(g, 6, W).abs() + 0.1, ref.rand(g, 6)
    dy = ref.rand(g, 1, T, 6, dtype=dtype)
    for t in range(T):
        bad = x.clone()
        bad[0, t, 2] = INF
        a = {"x": bad, "weight": w, "bias": b}
        want = ref.gradients(lambda **k: ref.conv(**k, act=None), ref.wide(a), list(a), (dy, None))
        got = gdn.gdn_conv_bwd(dy.cuda(), **ref.dev(a), act=None)
        long = torch.full((1, T + 6, 6), float("nan"), dtype=dtype)
        more = torch.full((1, T + 6, 6), float("nan"), dtype=dtype)
        long[:, :T], more[:, :T] = bad, dy
        pad = gdn.gdn_conv_bwd(more.cuda(), long.cuda(), w.cuda(), b.cuda(), lens=torch.tensor([T], dtype=torch.int32).cuda(),
                               act=None)
        for k in want:
            meets(f"d{k}, row {t}", got["d" + k], want[k])
            meets(f"d{k}, row {t}, padded", pad["d" + k][:, :T] if k == "x" else pad["d" + k], want[k])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 20, 70])
@pytest.mark.parametrize("N", [4, 7, 16, 32, 64])
@pytest.mark.parametrize("T,t", [(8, 5), (40, 21)])
@pytest.mark.parametrize("where", ["Bm", "C"])
def test_scan_gradient_of_part_of_a_wave(dtype, D, N, T, t, where):
    """Lanes without a channel add nothing to the sums over channels where B or
    C, which all lanes take, is infinite."""
    a = inputs(T, D, N, dtype, T)
    g = ref.gen(N)
    dy, dh = ref.rand(g, 1, T, D).abs().to(dtype), ref.rand(g, 1, D, N).abs()
    a[where][0, t, 0, N // 2] = INF
    check_gradient(a, dy, dh)
    check_gradient(a, dy, dh, T=T + 13)
