"""The operators together, as a layer uses them: the convolution into the delta
rule or the state space recurrence, the heads normalised and gated; prompts
and then tokens; in captured graphs and on other streams."""
import numpy as np
import pytest
import torch

import gated_delta_rule_13_amd as gdn
import oracle
from tests import layer_ref as ref
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def test_delta_rule_layer():
    """conv -> gdn_chunk_fwd -> norm, and the next tokens by conv step,
    gdn_recurrent_fwd, norm.  Each operator against its own 64-bit reference
    on the inputs it was given (the bf16 roundings between them are inputs)."""
    B, T, H, d, W = 2, 150, 3, 64, 4
    g = ref.gen(3)
    proj = ref.rand(g, B, T + 2, 3 * H * d, dtype=BF).cuda()
    w = {n: ref.rand(g, H * d, W, std=0.5).cuda() for n in "qkv"}
    z = ref.rand(g, B, T + 2, H, d, dtype=BF).cuda()
    weight = (1 + ref.rand(g, d, std=0.1)).cuda()
    alpha = torch.exp(-0.1 * torch.rand(B, H, T + 2, generator=g)).cuda()
    beta = torch.rand(B, H, T + 2, generator=g).cuda()
    part = {n: proj[:, :, i * H * d:(i + 1) * H * d] for i, n in enumerate("qkv")}

    def unit(x):
        return torch.nn.functional.normalize(x.float(), dim=-1).to(BF)

    heads, states = {}, {}
    for n in "qkv":
        heads[n], states[n] = gdn.gdn_conv_fwd(part[n][:, :T], w[n], heads=H)
        want, _ = ref.conv(part[n][:, :T].double().cpu(), w[n].double().cpu(), heads=H)
        ref.close(n, heads[n], want)
    q, k, v = unit(heads["q"]), unit(heads["k"]), heads["v"]
    O, S = gdn.gdn_chunk_fwd(q, k, v, alpha[:, :, :T].contiguous(), beta[:, :, :T].contiguous())
    y = gdn.gdn_norm_fwd(O.transpose(1, 2), weight, None, z[:, :T])
    ref.close("y", y, ref.norm(O.transpose(1, 2).double().cpu(), weight.double().cpu(), None, z[:, :T].double().cpu()))
    seen = [(q, k, v)]
    for t in (T, T + 1):
        new = {}
        for n in "qkv":
            new[n] = gdn.gdn_conv_step(part[n][:, t], w[n], None, states[n]).view(B, H, 1, d)
        q1, k1, v1 = unit(new["q"]), unit(new["k"]), new["v"]
        O1, S = gdn.gdn_recurrent_fwd(q1, k1, v1, alpha[:, :, t:t + 1].contiguous(), beta[:, :, t:t + 1].contiguous(),
                                      S, S_final=S)
        y1 = gdn.gdn_norm_fwd(O1.transpose(1, 2), weight, None, z[:, t:t + 1])
        seen.append((q1, k1, v1))
    qs, ks, vs = (torch.cat([s[i] for s in seen], 2) for i in range(3))
    Or, _ = oracle.recurrent(qs.cpu(), ks.cpu(), vs.cpu(), alpha.cpu(), beta.cpu())
    last = torch.from_numpy(np.ascontiguousarray(Or[:, :, -1:]))
    want = ref.norm(last.transpose(1, 2), weight.double().cpu(), None, z[:, -1:].double().cpu())
    # the delta rule's own tolerance (2e-3) and the rounding to bf16
    assert float((y1.double().cpu() - want).abs().max() / want.abs().max()) < 2e-3 + 2.0 ** -8
    # the convolution's tokens equal the prompt's kernel on the whole
    whole, _ = gdn.gdn_conv_fwd(part["v"], w["v"], heads=H)
    assert torch.equal(whole, vs)


def layer_args(seed, B=2, T=200, D=96, N=16, dtype=BF):
    g = ref.gen(seed)
    a = {"proj": ref.rand(g, B, T, 2 * D, dtype=dtype), "w": ref.rand(g, D, 4, std=0.5), "b": ref.rand(g, D, std=0.1),
         "dt": ref.rand(g, B, T, D, dtype=dtype, std=0.5), "A": -torch.exp(ref.rand(g, D, N, std=0.5)),
         "bc": ref.rand(g, B, T, 2, N, dtype=dtype), "D": 1 + ref.rand(g, D, std=0.1), "bias": ref.rand(g, D) - 3,
         "norm": 1 + ref.rand(g, 32, std=0.1), "dy": ref.rand(g, B, T, D // 32, 32, dtype=dtype)}
    return ref.dev(a)


def layer(a):
    """Forward and gradient of conv -> ssm -> norm with a gate."""
    D = a["w"].shape[0]
    x, z = a["proj"][:, :, :D], a["proj"][:, :, D:].unflatten(2, (-1, 32))
    Bm, C = a["bc"][:, :, :1], a["bc"][:, :, 1:]
    u, st = gdn.gdn_conv_fwd(x, a["w"], a["b"])
    s, h = gdn.gdn_ssm_fwd(u, a["dt"], a["A"], Bm, C, a["D"], None, a["bias"])
    y = gdn.gdn_norm_fwd(s.unflatten(2, (-1, 32)), a["norm"], None, z)
    gn = gdn.gdn_norm_bwd(a["dy"], s.unflatten(2, (-1, 32)), a["norm"], None, z)
    gs = gdn.gdn_ssm_bwd(gn["dx"].flatten(2), u, a["dt"], a["A"], Bm, C, a["D"], None, a["bias"])
    gc = gdn.gdn_conv_bwd(gs["dx"], x, a["w"], a["b"])
    return {"y": y, "h": h, "st": st, "dz": gn["dz"], "dnorm": gn["dweight"], **{"s" + k: v for k, v in gs.items()},
            **{"c" + k: v for k, v in gc.items()}}


def test_state_space_layer_and_its_gradient():
    """The whole chain in fp32 against autograd through the chained 64-bit
    references."""
    a = layer_args(1, B=1, T=90, D=64, dtype=F32)
    got = layer(a)
    w = ref.wide(a)
    D = 64

    def fn(proj, w_, b, dt, A, bc, D_, bias, norm):
        u, _ = ref.conv(proj[:, :, :D], w_, b)
        s, _ = ref.ssm(u, dt, A, bc[:, :, :1], bc[:, :, 1:], D_, None, bias)
        return ref.norm(s.unflatten(2, (-1, 32)), norm, None, proj[:, :, D:].unflatten(2, (-1, 32)))

    args = {"proj": w["proj"], "w_": w["w"], "b": w["b"], "dt": w["dt"], "A": w["A"], "bc": w["bc"], "D_": w["D"],
            "bias": w["bias"], "norm": w["norm"]}
    want = ref.gradients(fn, args, list(args), (a["dy"],))
    # three operators' errors add up along the chain
    three = 3.0
    for name, g in (("cdx", want["proj"][:, :, :D]), ("dz", want["proj"][:, :, D:].unflatten(2, (-1, 32))),
                    ("cdweight", want["w_"]), ("cdbias", want["b"]), ("sddt", want["dt"]), ("sdA", want["A"]),
                    ("sdB", want["bc"][:, :, :1]), ("sdC", want["bc"][:, :, 1:]), ("sdD", want["D_"]),
                    ("sddt_bias", want["bias"]), ("dnorm", want["norm"])):
        ref.close(name, got[name], g, three * float(g.abs().max()))


def test_captured_graph_replays():
    """Forward and gradient in one captured graph, replayed on new inputs with
    eager work between: every replay equals the eager result, bit for bit."""
    a = layer_args(2)
    others = [layer_args(s) for s in (3, 4, 5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(a)
    for o in others + others[:1]:
        want = layer(o)
        for k in a:
            a[k].copy_(o[k])
        graph.replay()
        torch.cuda.synchronize()
        layer(others[0])
        for k in want:
            assert torch.equal(out[k], want[k]), k


def test_two_graphs_at_once_and_streams():
    """Two captured graphs replayed on two streams at once share nothing; a
    call on a stream argument equals one on the current stream."""
    args = [layer_args(6), layer_args(7)]
    want = [layer(a) for a in args]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(a))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(o[k], w[k]) for k in w)
    a, s = args[0], streams[0]
    D = a["w"].shape[0]
    y, _ = gdn.gdn_conv_fwd(a["proj"][:, :, :D], a["w"], a["b"], stream=s)
    s.synchronize()
    assert torch.equal(y, gdn.gdn_conv_fwd(a["proj"][:, :, :D], a["w"], a["b"])[0])


def test_every_entry_on_another_stream():
    """Calls with a stream argument, while another stream is current: the same
    bits, and the outputs belong to that stream."""
    a = layer_args(9, T=70)
    D = a["w"].shape[0]
    x, z = a["proj"][:, :, :D], a["proj"][:, :, D:].unflatten(2, (-1, 32))
    Bm, C = a["bc"][:, :, :1], a["bc"][:, :, 1:]
    u, st = gdn.gdn_conv_fwd(x, a["w"], a["b"])
    s, h = gdn.gdn_ssm_fwd(u, a["dt"], a["A"], Bm, C, a["D"], None, a["bias"])
    heads = s.unflatten(2, (-1, 32))
    calls = [
        lambda **k: gdn.gdn_conv_fwd(x, a["w"], a["b"], **k),
        lambda **k: gdn.gdn_conv_bwd(u, x, a["w"], a["b"], **k),
        lambda **k: gdn.gdn_conv_step(x[:, 0], a["w"], a["b"], st.clone(), **k),
        lambda **k: gdn.gdn_ssm_fwd(u, a["dt"], a["A"], Bm, C, a["D"], None, a["bias"], **k),
        lambda **k: gdn.gdn_ssm_bwd(s, u, a["dt"], a["A"], Bm, C, a["D"], None, a["bias"], **k),
        lambda **k: gdn.gdn_ssm_step(u[:, 0], a["dt"][:, 0], a["A"], Bm[:, 0], C[:, 0], a["D"], None, a["bias"],
                                     h=h.clone(), **k),
        lambda **k: gdn.gdn_norm_fwd(heads, a["norm"], None, z, **k),
        lambda **k: gdn.gdn_norm_bwd(a["dy"], heads, a["norm"], None, z, **k),
    ]
    side = torch.cuda.Stream()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        got = call(stream=side)
        side.synchronize()
        flat = lambda r: list(r.values()) if isinstance(r, dict) else list(r) if isinstance(r, tuple) else [r]  # noqa: E731
        for g, w in zip(flat(got), flat(want)):
            assert torch.equal(g, w)


def test_not_a_number_stays_in_its_sequence():
    """NaN and infinity in one sequence's inputs reach that sequence's outputs
    only (and the parameters' gradients, which sum over all)."""
    a = layer_args(10, B=3, T=70)
    D = a["w"].shape[0]
    bad = dict(a, proj=a["proj"].clone(), dt=a["dt"].clone(), bc=a["bc"].clone())
    bad["proj"][1, 20] = float("nan")
    bad["bc"][1, 30] = float("inf")
    got, want = layer(bad), layer(a)
    for k in ("y", "h", "st", "dz", "sdx", "sddt", "sdB", "sdC", "cdx"):
        for i in (0, 2):
            assert torch.equal(got[k][i], want[k][i]), k
    assert not torch.isfinite(got["y"][1].float()).all()
    assert torch.equal(got["y"][1, :17], want["y"][1, :17])       # (rows before it, too)


def test_prompt_then_tokens_of_a_state_space_layer():
    """A padded batch's prompt, then tokens on the states it left: as the
    reference on each sequence's own tokens."""
    say("case: ssm layer, padded prompt then tokens")
    B, T, D, N, new = 3, 90, 64, 16, 4
    g = ref.gen(8)
    lens = torch.tensor([90, 17, 0], dtype=torch.int32)
    x = ref.rand(g, B, T + new, D)
    w, b = ref.rand(g, D, 4, std=0.5), ref.rand(g, D, std=0.1)
    dt, A, bias = ref.rand(g, B, T + new, D), -torch.exp(ref.rand(g, D, N)), ref.rand(g, D) - 3
    bc = ref.rand(g, B, T + new, 2, N)
    d = [v.cuda() for v in (x, w, b, dt, A, bias, bc)]
    X, Wt, Bi, DT, AA, BB, BC = d
    u, cs = gdn.gdn_conv_fwd(X[:, :T], Wt, Bi, lens=lens.cuda())
    y, h = gdn.gdn_ssm_fwd(u, DT[:, :T], AA, BC[:, :T, :1], BC[:, :T, 1:], dt_bias=BB, lens=lens.cuda())
    outs = []
    for i in range(new):
        t = T + i
        u1 = gdn.gdn_conv_step(X[:, t], Wt, Bi, cs)
        outs.append(gdn.gdn_ssm_step(u1, DT[:, t], AA, BC[:, t, :1], BC[:, t, 1:], dt_bias=BB, h=h))
    for i in range(B):
        n = int(lens[i])
        pick = lambda v: torch.cat([v[i:i + 1, :n], v[i:i + 1, T:]], 1).double()  # noqa: E731
        uu, _ = ref.conv(pick(x), w.double(), b.double())
        yy, hh = ref.ssm(uu, pick(dt), A.double(), pick(bc)[:, :, :1], pick(bc)[:, :, 1:], dt_bias=bias.double())
        two = 2.0 * float(yy.abs().max())
        ref.close("tokens", torch.stack([o[i] for o in outs])[None], yy[:, n:], two)
        ref.close("h", h[i:i + 1], hh, 2.0 * float(hh.abs().max()))
        if n:
            ref.close("prompt", y[i:i + 1, :n], yy[:, :n], two)
