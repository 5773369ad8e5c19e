"""The launches that large calls run, at small sizes that reach them: long tiles
of the convolution, long and many segments of the scan, several kept groups,
heads whose groups of lanes walk over many rows.  Each test first makes sure, by
the workspace it is asked for, that it runs what it is meant to.  References are
the formulas in 64 bits on the GPU, gradients by autograd through them."""
import ctypes

import pytest
import torch

import gated_delta_rule_13_amd as gdn
from gated_delta_rule_13_amd import _layer
from tests import layer_ref as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def lengths(g, B, T, special):
    """Lengths of a batch: the special ones, the others anywhere."""
    lens = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[:len(special)] = torch.tensor(special[:B], dtype=torch.int32)
    return lens


def live_rows(B, T, lens):
    if lens is None:
        return torch.ones(B, T, 1, dtype=torch.bool, device="cuda")
    return (torch.arange(T, device="cuda")[None] < lens[:, None])[..., None]


def silu(x):
    return x / (1 + torch.exp(-x))


def close(name, got, want):
    """layer_ref.close where the tensors are."""
    w = want.detach()
    assert tuple(got.shape) == tuple(w.shape), (name, tuple(got.shape), tuple(w.shape))
    top = float(w.abs().max())
    off = (got.double() - w).abs() - torch.finfo(got.dtype).eps / 2 * w.abs()
    worst = float(off.max()) - ref.FP32_TOL * top            # (NaN is no number below 0)
    assert worst <= 0, f"{name}: off by {worst:.3e} more than allowed (largest number {top:.3e})"


def up256(n):
    return (n + 255) // 256 * 256


# ---- convolution ----

def conv(x, weight, bias, state0, lens, act):
    """-> y [B,T,D], state_out"""
    B, T, D = x.shape
    W = weight.shape[1]
    live = live_rows(B, T, lens)
    rows = torch.cat([state0, torch.where(live, x, 0.0)], 1)
    p = bias + sum(weight[:, j] * rows[:, j:j + T] for j in range(W))
    y = torch.where(live, silu(p) if act else p, 0.0)
    at = (lens.long() if lens is not None else torch.full((B,), T, device="cuda"))[:, None] + torch.arange(W - 1, device="cuda")
    return y, rows.gather(1, at[..., None].expand(-1, -1, D))


def conv_tile(dtype, B, T, D, W):
    """Rows of dx to a wave, from the partial sums that the gradient keeps: one
    row of them for four tiles."""
    s = _layer._conv_shape(torch.empty(B, T, D, dtype=dtype, device="meta"), torch.empty(D, W, device="meta"), None, "silu")
    need = gdn.gdn_conv_bwd_workspace_bytes(s)
    for rows in (64, 32, 16, 8):
        tile = rows - (W - 1)
        if need == up256((B * -(-T // tile) + 3) // 4 * D * (W + 1) * 4):
            return tile
    raise AssertionError(need)


CONV = [  # rows, B, T, D, W, heads, act
    (16, 16, 47, 21888, 4, None, "silu"), (32, 4, 200, 37472, 4, 16, "silu"), (64, 6, 130, 60000, 4, None, None),
    (64, 6, 130, 60000, 2, 30, "silu"), (32, 4, 200, 37489, 3, None, "silu"), (64, 6, 130, 60002, 3, 2, "silu"),
    (16, 16, 47, 21889, 4, None, None),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,B,T,D,W,heads,act", CONV)
def test_convolution_gradient_tiles(dtype, rows, B, T, D, W, heads, act):
    """Rows in the middle of a tile, with nothing at its ends among them."""
    say(f"case: conv bwd {dtype} rows {rows} B{B} T{T} D{D} W{W} heads {heads} {act}")
    if dtype is F32:
        D = D // 2 if heads is None else D // 2 // heads * heads
    tile = conv_tile(dtype, B, T, D, W)
    assert tile == rows - (W - 1)
    g = generator(D + T)
    a = {"x": rand(g, B, T, D, dtype=dtype), "weight": rand(g, D, W, std=W ** -0.5), "bias": rand(g, D, std=0.2),
         "state0": rand(g, B, W - 1, D, dtype=dtype)}
    # lengths that end within a tile's middle rows, at its end and a token past them
    lens = lengths(g, B, T, [T, tile, tile + W, tile + W + 3, 5, 0])
    dy, ds = rand(g, B, T, D, dtype=dtype), rand(g, B, W - 1, D, dtype=dtype)
    live = live_rows(B, T, lens)
    a["x"] = torch.where(live, a["x"], NAN)
    leaves = {k: v.double().requires_grad_(True) for k, v in a.items()}
    y, st = conv(**leaves, lens=lens, act=act)
    want = torch.autograd.grad([y, st], list(leaves.values()), [torch.where(live, dy.double(), 0.0), ds.double()])
    dead = torch.where(live, dy, NAN)
    hd = dead if heads is None else dead.unflatten(2, (heads, -1)).transpose(1, 2).contiguous()
    got = gdn.gdn_conv_bwd(hd, **a, lens=lens, dstate_out=ds, act=act)
    for k, w in zip(leaves, want):
        close("d" + k, got["d" + k], w)
    out, state = gdn.gdn_conv_fwd(**a, lens=lens, heads=heads, act=act)
    out = out if heads is None else out.transpose(1, 2).flatten(2)
    close("y", out, y)
    assert torch.equal(state.double(), st)


# ---- scan ----

def scan_args(g, B, T, D, N, G, dtype, special):
    a = {"x": rand(g, B, T, D, dtype=dtype), "dt": rand(g, B, T, D, dtype=dtype, std=0.5),
         "A": -torch.arange(1, N + 1, device="cuda").float() * torch.exp(rand(g, D, N, std=0.2)),
         "Bm": rand(g, B, T, G, N, dtype=dtype), "C": rand(g, B, T, G, N, dtype=dtype), "D": 1 + rand(g, D, std=0.2),
         "z": rand(g, B, T, D, dtype=dtype), "dt_bias": rand(g, D) - 3, "h0": rand(g, B, D, N)}
    lens = lengths(g, B, T, special)
    live = live_rows(B, T, lens)
    for k in ("x", "dt", "z"):
        a[k] = torch.where(live, a[k], NAN)
    for k in ("Bm", "C"):
        a[k] = torch.where(live[..., None], a[k], NAN)
    return a, lens, live


def scan(x, dt, A, Bm, C, D, z, dt_bias, h0, live):
    """-> y, h"""
    G = Bm.shape[2]
    x, dt, z = (torch.where(live, v, 0.0) for v in (x, dt, z))
    s = torch.where(live, torch.logaddexp(dt + dt_bias, torch.zeros((), device="cuda", dtype=torch.float64)), 0.0)
    Bm, C = (torch.where(live[..., None], v, 0.0).repeat_interleave(x.shape[2] // G, dim=2) for v in (Bm, C))
    h, ys = h0, []
    for t in range(x.shape[1]):
        h = torch.exp(s[:, t, :, None] * A) * h + (s[:, t] * x[:, t])[..., None] * Bm[:, t]
        ys.append((h * C[:, t]).sum(-1))
    return torch.where(live, (torch.stack(ys, 1) + D * x) * silu(z), 0.0), h


def states(N):
    return next(n for n in (4, 8, 16, 32, 64) if N <= n)


def scan_shape(B, T, D, N, G):
    e = lambda *s: torch.empty(s, device="meta")  # noqa: E731
    return _layer._ssm_shape(e(B, T, D), e(B, T, D), e(D, N), e(B, T, G, N), e(B, T, G, N), None, True)


def forward_segments(B, T, D, N, G):
    need = gdn.gdn_ssm_fwd_workspace_bytes(scan_shape(B, T, D, N, G))
    return need // (B * G * -(-(D // G) // 64) * (states(N) + 1) * 64 * 4) if need else 1


def gradient_segment(B, T, D, N, G):
    """Tokens of a segment of the gradient, from its workspace."""
    need, ns, tiles = gdn.gdn_ssm_bwd_workspace_bytes(scan_shape(B, T, D, N, G)), states(N), G * -(-(D // G) // 64)
    for seg in (64, 32, 16):
        units = B * -(-T // seg) * tiles
        if need == units * 64 * 4 * (3 * ns + 3 + (seg // 8 - 1) * (ns + 1)) + up256(tiles * B * T * 2 * ns * 4):
            return seg
    raise AssertionError(need)


FORWARD = [  # segments, B, T, D, N, G
    (9, 4, 1000, 258, 16, 86), (9, 4, 1000, 258, 24, 86), (2, 20, 70, 258, 16, 86), (1, 36, 70, 258, 16, 86),
    (1, 36, 70, 258, 7, 86), (1, 36, 70, 258, 64, 86), (9, 2, 600, 6020, 4, 86), (36, 1, 1430, 4500, 16, 1),
    (36, 1, 1430, 4500, 3, 1),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("segments,B,T,D,N,G", FORWARD)
def test_scan_segments(dtype, segments, B, T, D, N, G):
    """Segments of more than 16 tokens, more of them than a chain has in
    flight, and prompts in one piece."""
    say(f"case: ssm fwd {dtype} {segments} segments B{B} T{T} D{D} N{N} G{G}")
    assert forward_segments(B, T, D, N, G) == segments
    per = -(-(-(-T // segments)) // 8) * 8
    assert segments == 1 or per > 16
    g = generator(T + N)
    a, lens, live = scan_args(g, B, T, D, N, G, dtype, [T, min(T, per + 9), per, 1] if B > 1 else [T - 3])
    y, h = gdn.gdn_ssm_fwd(**a, lens=lens)
    want, wh = scan(**{k: v.double() for k, v in a.items()}, live=live)
    close("y", y, want)
    close("h", h, wh)


GRADIENT = [  # segment, B, T, D, N, G
    (64, 16, 130, 1408, 4, 1), (64, 4, 130, 258, 16, 86), (64, 4, 130, 258, 7, 86), (64, 4, 130, 3010, 64, 43),
    (64, 4, 131, 258, 24, 86), (32, 4, 96, 258, 16, 86), (32, 4, 95, 258, 24, 86), (32, 4, 96, 258, 3, 86),
    (16, 1, 600, 20, 16, 1), (16, 2, 1100, 10, 7, 1), (64, 4, 2300, 30, 16, 10),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("segment,B,T,D,N,G", GRADIENT)
def test_scan_gradient_segments(dtype, segment, B, T, D, N, G):
    """Up to seven kept groups to a segment, and up to 69 segments."""
    say(f"case: ssm bwd {dtype} segment {segment} B{B} T{T} D{D} N{N} G{G}")
    assert gradient_segment(B, T, D, N, G) == segment
    g = generator(T + N)
    a, lens, live = scan_args(g, B, T, D, N, G, dtype, [T, T - 1, segment + 9, 8 * (segment // 16)] if B > 2 else [T, T // 2 + 3])
    dy, dh = rand(g, B, T, D, dtype=dtype), rand(g, B, D, N)
    leaves = {k: v.double().requires_grad_(True) for k, v in a.items()}
    out = scan(**leaves, live=live)
    want = torch.autograd.grad(out, list(leaves.values()), [torch.where(live, dy.double(), 0.0), dh.double()])
    got = gdn.gdn_ssm_bwd(torch.where(live, dy, NAN), **a, lens=lens, dh_final=dh)
    for k, w in zip(leaves, want):
        close("d" + k, got["dB" if k == "Bm" else "d" + k], w)


def test_rows_of_b_and_c_past_32_bits():
    """A token's B and C in rows more than 2^31 numbers apart."""
    g = generator(3)
    far = 2 ** 31 + 64
    memory = torch.empty(far + 64, dtype=BF, device="cuda")
    bm, c = (memory[i:].as_strided((2, 1, 16), (far, 16, 1)) for i in (0, 32))
    near = [rand(g, 2, 1, 16, dtype=BF) for _ in range(2)]
    bm.copy_(near[0])
    c.copy_(near[1])
    a = {"x": rand(g, 2, 40, dtype=BF), "dt": rand(g, 2, 40, dtype=BF), "A": -rand(g, 40, 16).abs()}
    h = rand(g, 2, 40, 16)
    h2 = h.clone()
    y = gdn.gdn_ssm_step(**a, Bm=bm, C=c, h=h)
    assert torch.equal(y, gdn.gdn_ssm_step(**a, Bm=near[0], C=near[1], h=h2)) and torch.equal(h, h2)


# ---- normalisation ----

def norm(x, weight, bias, z, center):
    c = x - x.mean(-1, keepdim=True) if center else x
    return (c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * weight + bias) * silu(z)


WALKS = [  # B, T, G, d: 8, 16, 32 and 64 lanes to a row, pieces of four and single numbers
    (3, 6701, 4, 128), (701, 143, 1, 24), (2, 3501, 8, 192), (911, 23, 3, 61), (1, 5003, 6, 512), (3, 4999, 2, 250),
    (2, 2203, 5, 1000), (1, 9001, 2, 500), (5, 2003, 3, 511), (7, 1501, 30, 96),
]


@pytest.mark.parametrize("xdt,odt", [(F32, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("B,T,G,d", WALKS)
def test_norm_walks(xdt, odt, B, T, G, d):
    """Groups of lanes that take several rows each, and not all of a wave the
    same number."""
    say(f"case: norm {xdt} -> {odt} B{B} T{T} G{G} d{d}")
    # more rows than four waves on each of the 1024 vector units take at once
    wide = d % 4 == 0
    lanes = next(n for n in (8, 16, 32, 64) if d <= n * (16 if wide else 8 if n > 8 else 4))
    assert B * T * G > 4096 * 64 // lanes * 1.2
    g = generator(T)
    x = rand(g, B, G, T, d, dtype=xdt).transpose(1, 2)
    w, b, z = 1 + rand(g, d, std=0.2), rand(g, d, std=0.2), rand(g, B, T, G, d, dtype=odt)
    dy = rand(g, B, T, G, d, dtype=odt)
    leaves = [v.double().requires_grad_(True) for v in (x, w, b, z)]
    y = norm(*leaves, True)
    want = torch.autograd.grad(y, leaves, dy.double())
    close("y", gdn.gdn_norm_fwd(x, w, b, z, center=True), y)
    got = gdn.gdn_norm_bwd(dy, x, w, b, z, center=True)
    for k, v in zip(("dx", "dweight", "dbias", "dz"), want):
        close(k, got[k], v)
