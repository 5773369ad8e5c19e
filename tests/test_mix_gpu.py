"""Linear attention and the norms around a block together, as a stack uses them:
norm of the stream, convolution, linear attention, head norm, and back into the
stream; with gradients, in captured graphs and on other streams, on far rows."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def block_args(seed, B=2, T=150, H=3, d=32, dtype=BF, stream=F32):
    g = ref.gen(seed)
    D = H * d
    a = {"o": ref.rand(g, B, T, D, dtype=dtype), "x": ref.rand(g, B, T, D, dtype=stream), "gate": ref.rand(g, B, T, D, dtype=dtype),
         "w_pre": 1 + ref.rand(g, D, std=0.2), "w_post": 1 + ref.rand(g, D, std=0.2), "scale": 0.5 + ref.rand(g, D, std=0.2),
         "conv": ref.rand(g, D, 4, std=0.5), "log_alpha": -0.1 * torch.rand(B, T, H, generator=g), "norm": 1 + ref.rand(g, d, std=0.2),
         "dx": ref.rand(g, B, T, D, dtype=stream), "dy": ref.rand(g, B, T, D, dtype=dtype)}
    return ref.dev(a)


def block(a):
    """The stream with a block's output, the next block on it (its queries, keys
    and values all the convolved stream), the stream behind that, and the gradient
    of all of it."""
    B, T, D = a["x"].shape
    H = a["log_alpha"].shape[2]
    d = D // H
    la = a["log_alpha"].transpose(1, 2)
    x1, y1 = gdn.gdn_block_norm_fwd(a["o"], a["x"], a["w_pre"], a["w_post"], a["gate"], a["scale"])
    u, _ = gdn.gdn_conv_fwd(y1, a["conv"], heads=H)
    o, S = gdn.gdn_lin_fwd(u, u, u, la, scale=d ** -0.5)
    n = gdn.gdn_norm_fwd(o.transpose(1, 2), a["norm"], act=None)
    x2, y2 = gdn.gdn_block_norm_fwd(n.flatten(2), x1, a["w_pre"], a["w_post"], a["gate"], a["scale"], act="silu")
    g2 = gdn.gdn_block_norm_bwd(a["dx"], a["dy"], x2, n.flatten(2), a["w_pre"], a["w_post"], a["gate"], a["scale"], act="silu")
    gn = gdn.gdn_norm_bwd(g2["do"].unflatten(2, (H, d)), o.transpose(1, 2), a["norm"], act=None)
    gl = gdn.gdn_lin_bwd(gn["dx"].transpose(1, 2).contiguous(), u, u, u, la, scale=d ** -0.5)
    gc = gdn.gdn_conv_bwd((gl["dq"].float() + gl["dk"].float() + gl["dv"].float()).to(u.dtype), y1, a["conv"])
    g1 = gdn.gdn_block_norm_bwd(g2["dx"], gc["dx"], x1, a["o"], a["w_pre"], a["w_post"], a["gate"], a["scale"])
    return {"x2": x2, "y2": y2, "S": S, "dconv": gc["dweight"], "dnorm": gn["dweight"], "dlog_alpha": gl["dlog_alpha"],
            **{"one_" + k: v for k, v in g1.items()}, **{"two_" + k: v for k, v in g2.items()}}


def test_two_blocks_and_their_gradient():
    """The whole chain in fp32 against autograd through the chained 64-bit
    references: six operators' errors add up, each within 1e-5 of a tensor's
    largest number (2^-16 of the terms of linear attention), and are carried
    through norms that keep their size."""
    a = block_args(1, B=1, T=90, dtype=F32)
    got = block(a)
    w = ref.wide(a)
    H, d = 3, 32

    def fn(o, x, gate, w_pre, w_post, scale, conv, log_alpha, norm):
        x1, y1 = mix.block(o, x, w_pre, w_post, gate, scale)
        u, _ = ref.conv(y1, conv, heads=H)
        att, _ = mix.lin(u, u, u, log_alpha.transpose(1, 2), scale=d ** -0.5)
        n = ref.norm(att.transpose(1, 2), norm, act=None)
        return mix.block(n.flatten(2), x1, w_pre, w_post, gate, scale, act="silu")

    names = ["o", "x", "gate", "w_pre", "w_post", "scale", "conv", "log_alpha", "norm"]
    args = {n: w[n] for n in names}
    x2, y2 = fn(**args)
    ref.close("x2", got["x2"], x2, 10.0 * float(x2.abs().max()))
    ref.close("y2", got["y2"], y2, 10.0 * float(y2.abs().max()))
    want = ref.gradients(fn, args, names, (a["dx"], a["dy"]))
    mine = {"o": got["one_do"], "x": got["one_dx"], "gate": got["one_dgate"] + got["two_dgate"], "conv": got["dconv"],
            "norm": got["dnorm"], "log_alpha": got["dlog_alpha"].transpose(1, 2),
            **{n: got["one_d" + n] + got["two_d" + n] for n in ("w_pre", "w_post", "scale")}}
    for n in names:
        ref.close(n, mine[n], want[n], 20.0 * float(want[n].abs().max()))


def test_captured_graph_replays():
    """Forward and gradient in one captured graph, replayed on new inputs with
    eager work between: every replay equals the eager result, bit for bit."""
    a = block_args(2)
    others = [block_args(s) for s in (3, 4, 5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(a)
    for o in others + others[:1]:
        want = block(o)
        for k in a:
            a[k].copy_(o[k])
        graph.replay()
        torch.cuda.synchronize()
        block(others[0])
        for k in want:
            assert torch.equal(out[k], want[k]), k


def test_two_graphs_at_once():
    """Two captured graphs with segments' workspaces, replayed on two streams at
    once, share nothing."""
    args = [block_args(s, B=1, T=700, H=2) for s in (6, 7)]
    want = [block(a) for a in args]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block(a))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(o[k], w[k]) for k in w)


def test_every_entry_on_another_stream():
    """Calls with a stream argument, while another stream is current: the same
    bits, and the outputs belong to that stream."""
    a = block_args(8, T=600, H=2)
    u = gdn.gdn_conv_fwd(a["x"].to(BF), a["conv"], heads=2)[0]
    la = a["log_alpha"].transpose(1, 2)
    S = torch.randn(2, 2, 32, 32, device="cuda")
    w = (a["w_pre"], a["w_post"], a["gate"], a["scale"])
    x1, _ = gdn.gdn_block_norm_fwd(a["o"], a["x"], *w)
    calls = [
        lambda **k: gdn.gdn_lin_fwd(u, u, u, la, S, **k),
        lambda **k: gdn.gdn_lin_bwd(u, u, u, u, la, S, dS_final=S, **k),
        lambda **k: gdn.gdn_lin_step(u[:, :, 0], u[:, :, 0], u[:, :, 0], la[:, :, 0], S.clone(), **k),
        lambda **k: gdn.gdn_block_norm_fwd(a["o"], a["x"], *w, **k),
        lambda **k: gdn.gdn_block_norm_bwd(a["dx"], a["dy"], x1, a["o"], *w, **k),
    ]
    side = torch.cuda.Stream()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        got = call(stream=side)
        side.synchronize()
        flat = lambda r: list(r.values()) if isinstance(r, dict) else list(r) if isinstance(r, tuple) else [r]  # noqa: E731
        for g, e in zip(flat(got), flat(want)):
            assert torch.equal(g, e)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_rows(dtype):
    """Sequences, heads and tokens more than 2^32 bytes apart, as dense copies."""
    say(f"case: far rows {dtype}")
    T, d = 70, 32
    far = torch.empty(2 ** 31 + 2 ** 22, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def place(*strides):
        t = far.as_strided((2, 2, T, d), (*strides, 1), storage_offset=place.at)
        place.at += 2 ** 16
        t.copy_(torch.randn(2, 2, T, d, generator=g, device="cuda"))
        return t
    place.at = 0
    # (sequences; heads; tokens 2^24 apart, past a chunk's 32-bit offsets)
    q, k = place(2 ** 31, T * d, d), place(T * d, 2 ** 31 + 64, d)
    v = far.as_strided((2, 2, T, d), (64, 32, 2 ** 24, 1), storage_offset=place.at)
    v.copy_(torch.randn(2, 2, T, d, generator=g, device="cuda"))
    la = -0.1 * torch.rand(2, 2, T, generator=g, device="cuda")
    views, dense = (q, k, v), [t.contiguous() for t in (q, k, v)]
    O, S = gdn.gdn_lin_fwd(*views, la)
    O1, S1 = gdn.gdn_lin_fwd(*dense, la)
    assert torch.equal(O, O1) and torch.equal(S, S1)
    x, y = gdn.gdn_lin_bwd(O, *views, la), gdn.gdn_lin_bwd(O, *dense, la)
    assert all(torch.equal(x[n], y[n]) for n in x)
    one = [t[:, :, 69] for t in views]
    A, B = S.clone(), S.clone()
    assert torch.equal(gdn.gdn_lin_step(*one, la[:, :, 69], A), gdn.gdn_lin_step(*[t.contiguous() for t in one], la[:, :, 69], B))
    assert torch.equal(A, B)
    o = q[:, 0]                                                   # sequences 2^31 elements apart
    x1, y1 = gdn.gdn_block_norm_fwd(o, o, gate=k[:, 1])
    x2, y2 = gdn.gdn_block_norm_fwd(o.contiguous(), o.contiguous(), gate=k[:, 1].contiguous())
    assert torch.equal(x1, x2) and torch.equal(y1, y2)


def test_what_lies_behind_outputs_stays():
    """Outputs of the caller's inside larger buffers: nothing around them is
    written."""
    a = block_args(9, T=77, H=2)
    u = gdn.gdn_conv_fwd(a["x"].to(BF), a["conv"], heads=2)[0]

    def guarded(shape, dtype):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[256:256 + n].view(shape)
    fO, O = guarded((2, 2, 77, 32), BF)
    fS, S = guarded((2, 2, 32, 32), F32)
    gdn.gdn_lin_fwd(u, u, u, a["log_alpha"].transpose(1, 2), lens=torch.tensor([77, 3], dtype=torch.int32, device="cuda"), O=O, S_final=S)
    fx, x = guarded((2, 77, 64), F32)
    fy, y = guarded((2, 77, 64), BF)
    gdn.gdn_block_norm_fwd(a["o"], a["x"], a["w_pre"], a["w_post"], a["gate"], a["scale"], x_out=x, y=y)
    for buf in (fO, fS, fx, fy):
        assert bool((buf[:256] == 7).all()) and bool((buf[-256:] == 7).all())
    assert not O[1, :, 3:].any()
    for t in (O, S, x, y):
        assert torch.isfinite(t.float()).all()
