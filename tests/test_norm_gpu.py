"""The normalisation of heads with an activation or a gate, on the GPU,
against the 64-bit reference."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, G, d, xdt, odt, seed, weight="d", gate=True, heads_first=False, bias=True):
    g = ref.gen(seed)
    x = ref.rand(g, B, G, T, d, dtype=xdt).transpose(1, 2) if heads_first else ref.rand(g, B, T, G, d, dtype=xdt)
    shape = {"d": (d,), "Gd": (G, d), None: None}[weight]
    return {"x": x, "weight": None if shape is None else 1 + ref.rand(g, *shape, std=0.3),
            "bias": None if shape is None or not bias else ref.rand(g, *shape, std=0.3),
            "z": ref.rand(g, B, T, G, d, dtype=odt) if gate else None}


def on_gpu(a):
    """Copies on the GPU that keep the strides."""
    out = ref.dev(a)
    if not a["x"].is_contiguous():
        out["x"] = a["x"].transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return out


CASES = [  # B, T, G, d, weight, gate, heads_first, center, act
    (1, 1, 1, 1, "d", True, False, False, "silu"), (2, 3, 2, 3, "Gd", False, False, True, "silu"),
    (1, 5, 3, 4, "d", True, True, False, None), (2, 1, 4, 64, "d", True, False, False, "silu"),
    (3, 7, 5, 96, "Gd", True, True, True, "silu"), (2, 33, 2, 128, "d", True, True, False, "silu"),
    (1, 70, 30, 192, "d", True, True, False, "silu"), (1, 9, 2, 256, None, False, False, True, None),
    (2, 5, 3, 250, "d", True, False, True, "silu"), (1, 4, 2, 512, "Gd", True, False, False, "silu"),
    (1, 3, 2, 1000, "d", False, True, False, "silu"), (1, 3, 2, 1024, "d", True, False, True, "silu"),
    (2, 2, 1, 2048, "d", True, False, False, "silu"), (1, 2, 2, 2052, "Gd", True, False, True, "silu"),
    (1, 2, 1, 4096, "d", True, False, False, "silu"), (1, 6, 2, 4095, None, True, False, False, "silu"),
    (2, 40, 2, 36, "d", True, False, False, "silu"), (1, 11, 7, 132, "Gd", True, False, True, "silu"),
]


@pytest.mark.parametrize("xdt,odt", [(F32, BF), (BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("B,T,G,d,weight,gate,heads_first,center,act", CASES)
def test_forward(xdt, odt, B, T, G, d, weight, gate, heads_first, center, act):
    say(f"case: norm fwd {xdt} -> {odt} B{B} T{T} G{G} d{d} {weight}")
    a = inputs(B, T, G, d, xdt, odt, d + T, weight, gate, heads_first)
    y = torch.full((B, T, G, d), float("nan"), dtype=odt, device="cuda")
    gdn.gdn_norm_fwd(**on_gpu(a), act=act, center=center, o_dtype=odt, y=y)
    ref.close("y", y, ref.norm(**ref.wide(a), act=act, center=center))


@pytest.mark.parametrize("xdt,odt", [(F32, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("B,T,G,d,weight,gate,heads_first,center,act", CASES + [(2, 700, 3, 24, "d", True, True, True, "silu"),
                                                                               (1, 1500, 2, 5, "Gd", False, False, False, "silu")])
def test_gradient(xdt, odt, B, T, G, d, weight, gate, heads_first, center, act):
    say(f"case: norm bwd {xdt} -> {odt} B{B} T{T} G{G} d{d} {weight}")
    a = inputs(B, T, G, d, xdt, odt, d + T, weight, gate, heads_first)
    dy = ref.rand(ref.gen(5), B, T, G, d, dtype=odt)
    d_ = on_gpu(a)
    got = gdn.gdn_norm_bwd(dy.cuda(), **d_, act=act, center=center)
    names = [n for n in ("x", "weight", "bias", "z") if a[n] is not None]
    want = ref.gradients(lambda **k: ref.norm(**k, act=act, center=center), ref.wide(a), names, (dy,))
    assert set(got) == {"d" + n for n in names}
    # (a row of d = 1 has the gradient r dp eps / (x^2 + eps): what is left
    # when two numbers near dp / |x| cancel)
    scale = {"x": float((dy.double() * (1 if a["z"] is None else 1)).abs().max()) / float(a["x"].double().abs().min())} if d == 1 else {}
    for n in names:
        ref.close("d" + n, got["d" + n], want[n], scale.get(n))
    again = gdn.gdn_norm_bwd(dy.cuda(), **d_, act=act, center=center)
    assert all(torch.equal(got[k], again[k]) for k in got)
    if heads_first:
        assert got["dx"].stride() == d_["x"].stride()


@pytest.mark.parametrize("xdt,odt", [(F32, BF), (BF, BF)])
@pytest.mark.parametrize("d", [7, 33, 63, 65, 97, 127, 129, 191, 193, 255, 257, 383, 385, 511, 513, 1023, 1025, 2047, 2049])
def test_odd_rows(xdt, odt, d):
    """Rows that no piece of four divides, at the ends of the kernels' ranges."""
    say(f"case: norm odd rows {xdt} -> {odt} d{d}")
    a = inputs(2, 5, 3, d, xdt, odt, d, "Gd", True, True)
    y = torch.full((2, 5, 3, d), float("nan"), dtype=odt, device="cuda")
    d_ = on_gpu(a)
    gdn.gdn_norm_fwd(**d_, center=True, y=y)
    ref.close("y", y, ref.norm(**ref.wide(a), center=True))
    dy = ref.rand(ref.gen(d + 1), 2, 5, 3, d, dtype=odt)
    got = gdn.gdn_norm_bwd(dy.cuda(), **d_, center=True)
    names = ("x", "weight", "bias", "z")
    want = ref.gradients(lambda **k: ref.norm(**k, center=True), ref.wide(a), names, (dy,))
    for n in names:
        ref.close("d" + n, got["d" + n], want[n])


@pytest.mark.parametrize("B,T,G,d", [(700, 3, 2, 64), (1, 5000, 1, 24), (5000, 1, 3, 21), (37, 61, 7, 128), (2, 900, 1, 2052)])
def test_walk_over_sequences(B, T, G, d):
    """Groups whose next row lies in a later sequence, or several on: sliced
    rows, as dense ones to the bit."""
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    wide = torch.randn(B, T + 2, G, d + 4, generator=g, device="cuda")
    x, z = wide[:, 1:-1, :, :d], torch.randn(B, G, T, d, generator=g, device="cuda").transpose(1, 2)
    w = torch.randn(d, generator=g, device="cuda")
    dense = (x.contiguous(), w, w, z.contiguous())
    y, want = gdn.gdn_norm_fwd(x, w, w, z), gdn.gdn_norm_fwd(*dense)
    ref.close("y", want, ref.norm(*[t.cpu().double() for t in dense]))
    assert torch.equal(y, want)
    a, b = gdn.gdn_norm_bwd(want, x, w, w, z), gdn.gdn_norm_bwd(want, *dense)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_strides_and_alignment():
    """Slices of wider rows, aligned or not, and a broadcast x: as dense ones.
    The kernels of unaligned rows sum in another order than the others, so the
    two agree within the tolerance, not to the bit."""
    a = inputs(2, 9, 3, 64, F32, F32, 3)
    want = ref.norm(**ref.wide(a))
    d = ref.dev(a)
    for off in (0, 4, 1, 3):
        w = torch.full((2, 9, 3 * 64 + 8), float("nan"), device="cuda")
        w[:, :, off:off + 192] = d["x"].flatten(2)
        x = w[:, :, off:off + 192].unflatten(2, (3, 64))
        ref.close("y", gdn.gdn_norm_fwd(x, d["weight"], d["bias"], d["z"]), want)
        g = gdn.gdn_norm_bwd(d["z"], x, d["weight"], d["bias"], d["z"])
        base = gdn.gdn_norm_bwd(d["z"], d["x"], d["weight"], d["bias"], d["z"])
        for k in g:
            ref.close(k, g[k], base[k].double().cpu())
    one = d["x"][:1].expand(2, -1, -1, -1)
    y = gdn.gdn_norm_fwd(one, d["weight"], d["bias"], d["z"])
    ref.close("y", y, ref.norm(**{**ref.wide(a), "x": a["x"][:1].double().expand(2, -1, -1, -1)}))
    g = gdn.gdn_norm_bwd(d["z"], one, d["weight"], d["bias"], d["z"])
    assert g["dx"].is_contiguous() and g["dx"].shape == one.shape


def test_zero_and_constant_rows():
    """A row of zeros, and a constant one that centring leaves empty: n = 0,
    no NaN, whatever eps."""
    x = torch.zeros(1, 2, 1, 128, device="cuda")
    x[0, 1] = 3.0
    b = torch.full((128,), 0.5, device="cuda")
    for center in (False, True):
        y = gdn.gdn_norm_fwd(x, None, b, center=center, eps=1e-12)
        g = gdn.gdn_norm_bwd(torch.ones_like(x), x, None, b, center=center, eps=1e-5)
        assert torch.isfinite(y).all() and all(torch.isfinite(v).all() for v in g.values())
        ref.close("y", y, ref.norm(x.double().cpu(), None, b.double().cpu(), center=center, eps=1e-12))


def test_gradient_against_differences():
    a = inputs(1, 5, 2, 12, F32, F32, 21, "Gd")
    g = ref.gen(1)
    dy = ref.rand(g, 1, 5, 2, 12)
    got = gdn.gdn_norm_bwd(dy.cuda(), **ref.dev(a), center=True)
    w = ref.wide(a)
    fn = lambda **k: ref.norm(**k, center=True)  # noqa: E731
    for n in ("x", "weight", "bias", "z"):
        v = ref.rand(g, *a[n].shape).double()
        want = ref.difference(fn, w, n, v, (dy,))
        mine = got["d" + n].double().cpu()
        slack = (ref.FP32_TOL + 1e-6) * float(mine.abs().max() * v.abs().sum())
        assert abs(float((mine * v).sum()) - want) <= slack, n


def test_refused_calls():
    a = ref.dev(inputs(2, 6, 3, 16, F32, F32, 2))
    bad = [
        (dict(x=a["x"][..., ::2]), ValueError), (dict(x=a["x"].half()), TypeError), (dict(x=a["x"][0]), ValueError),
        (dict(weight=a["weight"].to(BF)), TypeError), (dict(weight=a["weight"][:8]), ValueError),
        (dict(bias=torch.zeros(3, 16, device="cuda")), ValueError), (dict(z=a["z"].to(BF), o_dtype=F32), TypeError),
        (dict(z=a["z"][:, :5]), ValueError), (dict(eps=0.0), gdn.GdnError), (dict(eps=float("nan")), gdn.GdnError),
        (dict(act="gelu"), ValueError), (dict(y=a["x"]), ValueError), (dict(x=a["x"].cpu()), ValueError),
        (dict(o_dtype=torch.float16), TypeError),
    ]
    for kw, err in bad:
        with pytest.raises(err):
            gdn.gdn_norm_fwd(**{**a, **kw})
    big = torch.zeros(1, 1, 1, 4097, device="cuda")
    with pytest.raises(gdn.GdnError):
        gdn.gdn_norm_fwd(big)
    with pytest.raises(ValueError):
        gdn.gdn_norm_bwd(a["z"][:, :5].contiguous(), **a)
