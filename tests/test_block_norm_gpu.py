"""The norms around a block on the GPU, against the 64-bit reference.

Tolerance: half a step of an output's type and 1e-5 of a tensor's largest number
(every factor carries a few roundings of 2^-24, sums over a row or over rows at
most some tens more)."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def inputs(B, T, D, odt, xdt, seed, post=True, gate=True, scale=True, weights=True):
    g = ref.gen(seed)
    return {"o": ref.rand(g, B, T, D, dtype=odt), "x": ref.rand(g, B, T, D, dtype=xdt, std=2.0),
            "w_pre": 1 + ref.rand(g, D, std=0.3) if weights else None,
            "w_post": 1 + ref.rand(g, D, std=0.3) if weights and post else None,
            "gate": ref.rand(g, B, T, D, dtype=odt) if gate else None, "scale": 0.5 + ref.rand(g, D, std=0.3) if scale else None}


CASES = [  # B, T, D, post, gate's act, scale, weights
    (1, 1, 1, True, "sigmoid", True, True), (2, 3, 5, True, "silu", False, True), (1, 2, 64, False, "none", True, True),
    (3, 1, 65, True, None, True, False), (2, 7, 256, True, "sigmoid", True, True), (1, 9, 300, False, "silu", True, True),
    (2, 4, 513, True, "sigmoid", False, True), (1, 5, 1024, True, "sigmoid", True, True), (1, 3, 1025, True, "silu", True, True),
    (2, 5, 2048, True, "sigmoid", True, True), (1, 3, 2880, False, "silu", True, True), (1, 2, 4096, True, "none", False, False),
    (1, 2, 4097, True, "sigmoid", True, True), (1, 3, 8192, True, "sigmoid", True, True), (1, 2, 16384, True, "silu", True, True),
    (1, 2, 16383, True, "sigmoid", True, True), (2, 600, 36, True, "sigmoid", True, True), (1, 1500, 260, True, "silu", True, True),
]
TYPES = [(BF, F32), (BF, BF), (F32, F32), (F32, BF)]


@pytest.mark.parametrize("odt,xdt", TYPES)
@pytest.mark.parametrize("B,T,D,post,act,scale,weights", CASES)
def test_forward(odt, xdt, B, T, D, post, act, scale, weights):
    say(f"case: block fwd {odt} {xdt} B{B} T{T} D{D} {act}")
    gate = act != "none"
    a = inputs(B, T, D, odt, xdt, D, post, gate, scale, weights)
    act = act if gate else None
    xo = torch.full((B, T, D), float("nan"), dtype=xdt, device="cuda")
    y = torch.full((B, T, D), float("nan"), dtype=odt, device="cuda")
    gdn.gdn_block_norm_fwd(**ref.dev(a), act=act, post=post, x_out=xo, y=y)
    wx, wy = mix.block(**ref.wide(a), act=act, post=post)
    ref.close("x_out", xo, wx)
    ref.close("y", y, wy)
    x2, none = gdn.gdn_block_norm_fwd(**{**ref.dev(a), "w_pre": None}, act=act, post=post, pre=False)
    assert none is None and torch.equal(x2, xo)


@pytest.mark.parametrize("odt,xdt", TYPES)
@pytest.mark.parametrize("B,T,D,post,act,scale,weights", CASES)
@pytest.mark.parametrize("part", ["both", "dx_out", "dy"])
def test_gradient(odt, xdt, B, T, D, post, act, scale, weights, part):
    say(f"case: block bwd {odt} {xdt} B{B} T{T} D{D} {act} {part}")
    gate = act != "none"
    a = inputs(B, T, D, odt, xdt, D, post, gate, scale, weights)
    act = act if gate else None
    g = ref.gen(D + 1)
    dx, dy = ref.rand(g, B, T, D, dtype=xdt), ref.rand(g, B, T, D, dtype=odt)
    if part == "dx_out":
        dy, a["w_pre"] = None, None
    elif part == "dy":
        dx = None
    # the stream behind the block is an input here, as it was stored
    w = ref.wide(a)
    xo = mix.block(**w, act=act, post=post)[0].to(xdt)
    names = [n for n in ("o", "w_post", "gate", "scale") if a[n] is not None]
    leaves = {n: w[n].clone().requires_grad_(True) for n in names}
    stored = xo.double().requires_grad_(True)
    wp = w["w_pre"].clone().requires_grad_(True) if a["w_pre"] is not None else None
    y = stored / torch.sqrt((stored * stored).mean(-1, keepdim=True) + 1e-5)
    y = y if wp is None else y * wp
    total = torch.zeros(B, T, D, dtype=torch.float64)
    want = {}
    if dy is not None:
        grads = torch.autograd.grad((y * dy.double()).sum(), [stored] + ([wp] if wp is not None else []))
        total = total + grads[0]
        if wp is not None:
            want["dw_pre"] = grads[1]
    if dx is not None:
        total = total + dx.double()
    want["dx"] = total
    n, _ = mix.block(**{**w, **leaves}, act=act, post=post)
    want.update({"d" + k: v for k, v in zip(names, torch.autograd.grad((n * total).sum(), list(leaves.values())))})
    d = ref.dev(a)
    d.pop("x")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    call = lambda: gdn.gdn_block_norm_bwd(cu(dx), cu(dy), xo.cuda(), **d, act=act, post=post)  # noqa: E731
    got = call()
    assert set(got) == set(want)
    # (a row of one number has the gradient r d eps / (x^2 + eps): what is left
    # when two numbers near d / |x| cancel; dx and what follows from it)
    scale_of = {}
    if D == 1:
        top = 10 * (1 + float(1 / xo.double().abs().min())) * (1 + float(1 / w["o"].abs().min()))
        scale_of = {k: top for k in want}
    for k in want:
        ref.close(k, got[k], want[k], scale_of.get(k))
    again = call()
    assert all(torch.equal(got[k], again[k]) for k in got)


def same(got, want, exact):
    """Equal bits where the same kernel ran; rows off their places run another,
    whose sums have another order: each within half a step and 1e-5 of the exact
    number, so the two within twice that."""
    if exact:
        return torch.equal(got, want)
    g, w = got.double(), want.double()
    return bool(((g - w).abs() <= torch.finfo(got.dtype).eps * w.abs() * (1 + 2.0 ** -7) + 2e-5 * w.abs().max()).all())


@pytest.mark.parametrize("odt,xdt", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("D,off", [(96, 4), (96, 1), (1500, 2), (33, 0)])
def test_views(odt, xdt, D, off):
    """Slices of wider rows, a gate that a sequence's tokens share, in place:
    as dense copies."""
    B, T = 2, 9
    g = ref.gen(D + off)
    wide = ref.rand(g, B, T, 2 * D + 8, dtype=odt).cuda()
    o, gate = wide[:, :, off:off + D], wide[:, :1, D + 4:2 * D + 4].expand(B, T, D)
    x = ref.rand(g, T, B, D + 4, dtype=xdt).cuda().transpose(0, 1)[:, :, :D]
    w = [1 + ref.rand(g, D, std=0.3).cuda() for _ in range(3)]
    want = gdn.gdn_block_norm_fwd(o.contiguous(), x.contiguous(), w[0], w[1], gate.contiguous(), w[2])
    got = gdn.gdn_block_norm_fwd(o, x, w[0], w[1], gate, w[2])
    ref.close("x", got[0], mix.block(*[t.double().cpu() for t in (o, x, w[0], w[1], gate, w[2])])[0])
    exact = off % 4 == 0
    assert same(got[0], want[0], exact) and same(got[1], want[1], exact)
    inplace = x.contiguous().clone()
    gdn.gdn_block_norm_fwd(o, inplace, w[0], w[1], gate, w[2], x_out=inplace)
    assert same(inplace, want[0], exact)
    dx, dy = ref.rand(g, B, T, D, dtype=xdt).cuda(), ref.rand(g, B, T, D, dtype=odt).cuda()
    xo = want[0].transpose(0, 1).contiguous().transpose(0, 1)
    a = gdn.gdn_block_norm_bwd(dx, dy, xo, o, w[0], w[1], gate, w[2])
    b = gdn.gdn_block_norm_bwd(dx, dy, want[0], o.contiguous(), w[0], w[1], gate.contiguous(), w[2])
    assert all(same(a[k], b[k], exact) for k in a)


def test_gates_at_the_ends_and_rows_of_zeros():
    """Infinite gates are their limits; a row of zeros stays one."""
    B, T, D = 1, 4, 64
    o, x = torch.randn(B, T, D, device="cuda"), torch.randn(B, T, D, device="cuda")
    gate = torch.zeros(B, T, D, device="cuda")
    gate[0, 0], gate[0, 1] = float("inf"), float("-inf")
    o[0, 2], x[0, 2] = 0, 0
    xo, y = gdn.gdn_block_norm_fwd(o, x, gate=gate)
    n = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-5)
    assert torch.allclose(xo[0, 0], x[0, 0] + n[0, 0], atol=1e-5) and torch.equal(xo[0, 1], x[0, 1])
    assert not xo[0, 2].any() and not y[0, 2].any() and torch.isfinite(y).all()
    g = gdn.gdn_block_norm_bwd(torch.ones_like(x), torch.ones_like(x), xo, o, gate=gate)
    assert all(torch.isfinite(v).all() for v in g.values()) and not g["dgate"][0, :2].any()
    # NaN stays in its row
    o2 = o.clone()
    o2[0, 3, 5] = float("nan")
    again, _ = gdn.gdn_block_norm_fwd(o2, x, gate=gate)
    assert torch.equal(again[0, :3], xo[0, :3]) and torch.isnan(again[0, 3]).all()
