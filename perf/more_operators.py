"""Linear attention with decay and the norms around a block: what each computes and how large it is in use.

In a stack of mixing layers, blocks of linear attention stand beside blocks of the gated delta rule (the same state,
without the erasing), and every block is joined to the residual stream by a norm, a gate and a scale. Two operators:

  lin    S_t = alpha_t S_{t-1} + v_t k_t^T, o_t = scale S_t q_t for each head, alpha_t = exp(log_alpha_t) for each head and
         token, or fixed for each head; S [d_v, d_k]. For prompts, for single tokens, and the gradient. Heads of values
         may share a head of queries or keys. `lens` holds each sequence's length in a batch padded to T tokens: what lies
         behind it reaches nothing, and outputs and gradients there are zero. log_alpha of minus infinity starts anew.
  block  x' = x + s act(g) n with n = o / sqrt(mean(o^2) + eps) w_post, and y = x' / sqrt(mean(x'^2) + eps) w_pre over the
         last dimension: o is a block's output, x the residual stream, g the block's gate, s a scale for each channel;
         y is what the next block reads. Forward and gradient.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
CHUNK = 64


def listed():
    def lin(name, op, **k):
        c = {"name": name, "op": op, "dtype": "bf16", "Hq": k["H"], "Hk": k["H"], "dk": 128, "dv": 128, "decay": "token",
             "resets": False, "lens": False, "state": False, **k}
        return c

    def block(name, op, **k):
        return {"name": name, "op": op, "dtype": "bf16", "xdtype": "f32", "post": True, "gate": "sigmoid", "scale": True, **k}

    return [
        # prompts of a batch through 16 heads of 128
        lin("lin prompts", "lin_fwd", B=4, H=16, T=4096),
        # one long prompt through few heads, each with a fixed decay: the length has to give the parallel work
        lin("lin long", "lin_fwd", B=1, H=8, T=32768, decay="head"),
        # many short prompts, narrow heads
        lin("lin many short", "lin_fwd", B=32, H=16, T=256, dk=64, dv=64, state=True),
        # odd sizes: padded prompts of packed documents in 32 bits, six heads of values on two of queries and keys
        lin("lin ragged f32", "lin_fwd", B=3, H=6, Hq=2, Hk=2, T=1021, dk=72, dv=40, dtype="f32", resets=True, lens=True,
            state=True),
        # one decode step of 64 sequences
        lin("lin token", "lin_step", B=64, H=16, T=1, state=True),
        # one decode step of one sequence, 30 heads of 96 and 192
        lin("lin token small", "lin_step", B=1, H=30, T=1, dk=96, dv=192, state=True),
        # the training step's gradient at the shape of the first case
        lin("lin gradient", "lin_bwd", B=4, H=16, T=4096),
        # a padded batch's gradient, eight heads of values on four of queries and keys, from a state and back to it
        lin("lin gradient ragged", "lin_bwd", B=2, H=8, Hq=4, Hk=4, T=777, dk=64, dv=128, lens=True, state=True),
        # a block's output into the residual stream and on to the next block's input, in training
        block("block prompts", "block_fwd", B=4, T=4096, D=2048),
        # the same for one token of 64 sequences
        block("block token", "block_fwd", B=64, T=1, D=2048, xdtype="bf16"),
        # the training step's gradient at the shape of the first
        block("block gradient", "block_bwd", B=4, T=4096, D=2048),
        # 2880 channels, all in 32 bits, a scale and a silu gate but no norm after the block
        block("block gradient f32", "block_bwd", B=2, T=1031, D=2880, dtype="f32", post=False, gate="silu"),
    ]


def _between(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_fwd", "lin_fwd", "lin_step", "lin_step", "lin_bwd", "lin_bwd", "block_fwd", "block_fwd",
                     "block_bwd", "block_bwd"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("block"):
        D = _between(rng, 64, 8192)
        rows = max(1, min(_between(rng, 1, 32768), (32 << 20) // D))
        B = rng.choice([1, 1, 2, 3])
        return {**c, "xdtype": rng.choice(["bf16", "f32"]), "B": B, "T": max(1, rows // B), "D": D, "post": rng.random() < 0.7,
                "gate": rng.choice(["none", "sigmoid", "silu"]), "scale": rng.random() < 0.6}
    one = op == "lin_step"
    shared = rng.choice([1, 1, 2, 3])
    Hq, Hk = rng.choice([(1, 1), (1, 1), (1, shared), (shared, 1)])
    groups = _between(rng, 1, 16)
    H = groups * Hq * Hk
    c.update(B=_between(rng, 1, 64 if one else 8), H=H, Hq=H // Hq, Hk=H // Hk)
    dims = [16, 32, 64, 64, 96, 128, 128, 256, _between(rng, 8, 256)]
    c.update(dk=rng.choice(dims), dv=rng.choice(dims), decay=rng.choice(["token", "token", "token", "head", "none"]))
    c["resets"] = c["decay"] == "token" and rng.random() < 0.3
    most = (1 << 32) // (c["B"] * H * max(c["dk"], 64) * max(c["dv"], 64))
    if op == "lin_bwd":
        most //= 2
    c["T"] = 1 if one else max(1, min(_between(rng, 1, 16384), most))
    return {**c, "lens": not one and rng.random() < 0.4, "state": one or rng.random() < 0.5}


def prepare(case, seed):
    op, dev = case["op"], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, T, dt = case["B"], case["T"], DTYPES[case["dtype"]]

    def rnd(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"op": op, "case": dict(case)}
    if op.startswith("block"):
        D, xdt = case["D"], DTYPES[case["xdtype"]]
        s["o"] = rnd(B, T, D, std=0.5, dtype=dt)
        # the gate is half of a wider projection's output
        s["gate"] = rnd(B, T, D + 8, dtype=dt)[:, :, 8:] if case["gate"] != "none" else None
        s["w_post"] = 1.0 + rnd(D, std=0.1) if case["post"] else None
        s["scale"] = 0.5 + rnd(D, std=0.1) if case["scale"] else None
        s["w_pre"] = 1.0 + rnd(D, std=0.1)
        # the stream before the block, or in the gradient behind it
        s["x"] = rnd(B, T, D, std=2.0, dtype=xdt)
        if op == "block_bwd":
            s["dx_out"] = rnd(B, T, D, dtype=xdt)
            s["dy"] = rnd(B, T, D, dtype=dt)
        return s
    H, Hq, Hk, dk, dv = case["H"], case["Hq"], case["Hk"], case["dk"], case["dv"]

    def unit(*shape):
        x = rnd(*shape)
        return (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)).to(dt)

    # queries, keys and values are slices of one projection's output
    parts = [unit(B, T, Hq, dk).flatten(2), unit(B, T, Hk, dk).flatten(2), rnd(B, T, H, dv, dtype=dt).flatten(2)]
    proj = torch.cat(parts, 2)
    at = 0
    for name, heads, d in (("q", Hq, dk), ("k", Hk, dk), ("v", H, dv)):
        s[name] = proj[:, :, at:at + heads * d].unflatten(2, (heads, d)).transpose(1, 2)
        at += heads * d
    if case["decay"] == "token":
        # memories of some 30 tokens
        la = -0.05 * torch.nn.functional.softplus(rnd(B, T, H))
        if case["resets"]:
            # documents packed into a row: some 200 tokens each
            la = torch.where(torch.rand(B, T, H, generator=g, device=dev) < 0.005, -math.inf, la)
        s["log_alpha"] = la.transpose(1, 2)
    else:
        # memories of 2 to 512 tokens, spread over the heads
        slopes = -torch.exp2(-9.0 * torch.rand(H, generator=g, device=dev))
        s["log_alpha"] = slopes if case["decay"] == "head" else None
    s["attn_scale"] = dk ** -0.5 * 4.0
    if case["lens"]:
        lens = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        lens[0] = T
        s["lens"] = lens
    if case["state"]:
        s["S0"] = rnd(B, H, dv, dk, std=0.3)
    if op == "lin_bwd":
        s["dO"] = rnd(B, H, T, dv, dtype=dt)
        if case["state"]:
            s["dS"] = rnd(B, H, dv, dk, std=0.3)
    if op == "lin_step":
        for n in "qkv":
            s[n] = s[n][:, :, 0]
        if case["decay"] == "token":
            s["log_alpha"] = s["log_alpha"][:, :, 0]
    return s


def run(s):
    if own:
        return _own(s)
    return {"lin_fwd": _lin_fwd, "lin_step": _lin_step, "lin_bwd": _lin_bwd, "block_fwd": _block_fwd, "block_bwd": _block_bwd}[s["op"]](s)


def _own(s):
    import gated_delta_rule_13_amd as gdn
    op, c = s["op"], s["case"]
    if op == "lin_fwd":
        O, S = gdn.gdn_lin_fwd(s["q"], s["k"], s["v"], s["log_alpha"], s.get("S0"), lens=s.get("lens"), scale=s["attn_scale"])
        return {"O": O, "S": S}
    if op == "lin_step":
        O = gdn.gdn_lin_step(s["q"], s["k"], s["v"], s["log_alpha"], s["S0"], scale=s["attn_scale"])
        return {"O": O, "S": s["S0"]}
    if op == "lin_bwd":
        return gdn.gdn_lin_bwd(s["dO"], s["q"], s["k"], s["v"], s["log_alpha"], s.get("S0"), lens=s.get("lens"),
                               dS_final=s.get("dS"), scale=s["attn_scale"])
    act = None if c["gate"] == "none" else c["gate"]
    if op == "block_fwd":
        x, y = gdn.gdn_block_norm_fwd(s["o"], s["x"], s["w_pre"], s["w_post"], s["gate"], s["scale"], act=act, post=c["post"], eps=EPS)
        return {"x": x, "y": y}
    return gdn.gdn_block_norm_bwd(s["dx_out"], s["dy"], s["x"], s["o"], s["w_pre"], s["w_post"], s["gate"], s["scale"], act=act,
                                  post=c["post"], eps=EPS)


def _chunks(x, n):
    """[B, H, T, ...] -> [B, H, n, CHUNK, ...], zeros behind the last token."""
    B, H, T = x.shape[:3]
    full = x.new_zeros(B, H, n * CHUNK, *x.shape[3:])
    full[:, :, :T] = x
    return full.unflatten(2, (n, CHUNK))


def _lin_parts(s):
    """Queries, keys, values by chunks in 32 bits for every head of values; the decays between tokens of a chunk [.., r, i]
    (0 for i > r), from a chunk's start and to its end, and over the whole of it."""
    q, k, v = (s[n].float() for n in "qkv")
    B, H, T, _ = v.shape
    q, k = q.repeat_interleave(H // q.shape[1], 1), k.repeat_interleave(H // k.shape[1], 1)
    la = s["log_alpha"]
    if la is None:
        la = torch.zeros(H, device=v.device)
    la = (la if la.dim() == 3 else la[None, :, None].expand(B, H, T)).double()
    if "lens" in s:
        live = (torch.arange(T, device=v.device) < s["lens"][:, None])[:, None, :]
        q, k, v = (torch.where(live[..., None], x, 0.0) for x in (q, k, v))
        la = torch.where(live, la, 0.0)
    n = -(-T // CHUNK)
    # (-1e4 is as good as minus infinity, and its differences are numbers)
    G = _chunks(la.clamp(min=-1e4), n).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    between = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    return (_chunks(q, n), _chunks(k, n), _chunks(v, n), between, G.exp().float(), (G[..., -1:] - G).exp().float(),
            G[..., -1].exp().float())


def _chain(whole, add, first):
    """States before each chunk, and behind the last: S <- whole S + add."""
    S, out = first, []
    for c in range(add.shape[2]):
        out.append(S)
        S = whole[:, :, c, None, None] * S + add[:, :, c]
    return torch.stack(out, 2), S


def _lin_states(s, k, v, to_end, whole):
    B, H = k.shape[:2]
    first = s["S0"].float() if "S0" in s else k.new_zeros(B, H, v.shape[-1], k.shape[-1])
    return _chain(whole, (v * to_end[..., None]).transpose(-1, -2) @ k, first)


def _lin_fwd(s):
    q, k, v, between, start, to_end, whole = _lin_parts(s)
    T, dt = s["v"].shape[2], s["v"].dtype
    S, last = _lin_states(s, k, v, to_end, whole)
    o = (q @ k.transpose(-1, -2) * between) @ v + start[..., None] * (q @ S.transpose(-1, -2))
    return {"O": (s["attn_scale"] * o).flatten(2, 3)[:, :, :T].to(dt).contiguous(), "S": last}


def _lin_step(s):
    q, k, v = (s[n].float() for n in "qkv")
    B, H = v.shape[:2]
    q, k = q.repeat_interleave(H // q.shape[1], 1), k.repeat_interleave(H // k.shape[1], 1)
    S = s["S0"]
    if s["log_alpha"] is not None:
        S = torch.exp(s["log_alpha"])[..., None, None] * S
    S = S + v[..., :, None] * k[..., None, :]
    s["S0"].copy_(S)
    return {"O": (s["attn_scale"] * (S * q[..., None, :]).sum(-1)).to(s["v"].dtype), "S": s["S0"]}


def _lin_bwd(s):
    q, k, v, between, start, to_end, whole = _lin_parts(s)
    B, H, n = q.shape[:3]
    T, dt, scale = s["v"].shape[2], s["v"].dtype, s["attn_scale"]
    do = s["dO"].float()
    if "lens" in s:
        do = torch.where((torch.arange(T, device=do.device) < s["lens"][:, None])[:, None, :, None], do, 0.0)
    do = _chunks(do, n) * scale
    S, last = _lin_states(s, k, v, to_end, whole)
    # the gradient of the state behind each chunk, from the last to the first
    add = (do * start[..., None]).transpose(-1, -2) @ q
    end = s["dS"].float() if "dS" in s else torch.zeros_like(last)
    D, dS0 = _chain(whole.flip(2), add.flip(2), end)
    D = D.flip(2)
    dA = do @ v.transpose(-1, -2) * between
    A = q @ k.transpose(-1, -2) * between
    dq = dA @ k + start[..., None] * (do @ S)
    dk = dA.transpose(-1, -2) @ q + to_end[..., None] * (v @ D)
    dv = A.transpose(-1, -2) @ do + to_end[..., None] * (k @ D.transpose(-1, -2))
    dq, dk, dv, q, k = (x.flatten(2, 3)[:, :, :T] for x in (dq, dk, dv, q, k))
    out = {"dv": dv.to(dt).contiguous()}
    out["dq"] = dq.unflatten(1, (s["q"].shape[1], -1)).sum(2).to(dt)
    out["dk"] = dk.unflatten(1, (s["k"].shape[1], -1)).sum(2).to(dt)
    if s["log_alpha"] is not None:
        # the state's share of the loss behind each token, and what later tokens took and earlier ones gave
        own_part = (q.double() * dq).sum(-1) - (k.double() * dk).sum(-1)
        g = own_part.flip(-1).cumsum(-1).flip(-1) + (end.double() * last).sum((-1, -2))[..., None]
        if "lens" in s:
            g = torch.where((torch.arange(T, device=g.device) < s["lens"][:, None])[:, None, :], g, 0.0)
        if s["log_alpha"].dim() == 1:
            g = g.sum((0, 2))
        else:
            g = torch.where(torch.isinf(s["log_alpha"]), 0.0, g)
        out["dlog_alpha"] = g.float()
    if "S0" in s:
        out["dS0"] = dS0
    return out


def _gate(s):
    """act(g) and act'(g)."""
    if s["gate"] is None:
        return 1.0, None
    g = s["gate"].float()
    e = 1.0 / (1.0 + torch.exp(-g))
    if s["case"]["gate"] == "sigmoid":
        return e, e * (1.0 - e)
    return g * e, e * (1.0 + g * (1.0 - e))


def _unit_rms(x):
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _block_fwd(s):
    n = s["o"].float()
    if s["case"]["post"]:
        n = _unit_rms(n)[0] * s["w_post"]
    a = _gate(s)[0] * n
    if s["scale"] is not None:
        a = a * s["scale"]
    x = s["x"].float() + a
    return {"x": x.to(s["x"].dtype), "y": (_unit_rms(x)[0] * s["w_pre"]).to(s["o"].dtype)}


def _block_bwd(s):
    post, scale = s["case"]["post"], s["scale"] if s["scale"] is not None else 1.0
    xh, r = _unit_rms(s["x"].float())
    dy = s["dy"].float()
    dn = dy * s["w_pre"]
    dx = s["dx_out"].float() + r * (dn - xh * (dn * xh).mean(-1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype), "dw_pre": (dy * xh).sum((0, 1))}
    o = s["o"].float()
    oh, r = _unit_rms(o) if post else (o, 1.0)
    n = oh * s["w_post"] if post else o
    act, slope = _gate(s)
    if s["scale"] is not None:
        out["dscale"] = (dx * act * n).sum((0, 1))
    if slope is not None:
        out["dgate"] = (dx * scale * n * slope).to(s["gate"].dtype)
    dn = dx * scale * act
    if post:
        out["dw_post"] = (dn * oh).sum((0, 1))
        dn = dn * s["w_post"]
        dn = r * (dn - oh * (dn * oh).mean(-1, keepdim=True))
    out["do"] = dn.to(s["o"].dtype)
    return out


def work(case):
    op, B, T = case["op"], case["B"], case["T"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("block"):
        n, xe = B * T * case["D"], 2 if case["xdtype"] == "bf16" else 4
        gate = e if case["gate"] != "none" else 0
        if op == "block_fwd":
            # o, gate, x read, x', y written
            return {"bytes": n * (2 * e + gate + 2 * xe), "flops": n * 20}
        # o, gate, x', their gradients, and dx_out, dy
        return {"bytes": n * (3 * e + 2 * gate + 3 * xe), "flops": n * 45}
    H, Hq, Hk, dk, dv = case["H"], case["Hq"], case["Hk"], case["dk"], case["dv"]
    tokens, state = B * T, B * H * dv * dk * 4
    ins = tokens * (Hq * dk + Hk * dk + H * dv) * e
    decay = tokens * H * 4 if case["decay"] == "token" else 0
    row = tokens * H * dv * e
    if op == "lin_bwd":
        # q, k, v, log_alpha and their gradients, dO; states, their gradients
        return {"bytes": 2 * ins + 2 * decay + row + (3 * state if case["state"] else 0), "flops": tokens * H * 10 * dk * dv}
    return {"bytes": ins + decay + row + state * (2 if case["state"] else 1), "flops": tokens * H * 4 * dk * dv}


def exact(case, seed):
    """The operators from their definitions in 64 bits, a token at a time where they are recurrences."""
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    if case["op"].startswith("block"):
        return _exact_block(case, s)
    H, T, step = case["H"], case["T"], case["op"] == "lin_step"
    wide = lambda x: x[:, torch.arange(H, device=x.device) // (H // x.shape[1])]  # noqa: E731
    q, k, v = wide(s["q"]), wide(s["k"]), s["v"]
    if step:
        q, k, v = q[:, :, None], k[:, :, None], v[:, :, None]
    B, dev = v.shape[0], v.device
    alpha = torch.ones(B, H, T, dtype=torch.float64, device=dev)
    if case["decay"] == "token":
        alpha = torch.exp(s["log_alpha"] if not step else s["log_alpha"][:, :, None])
    elif case["decay"] == "head":
        alpha = alpha * torch.exp(s["log_alpha"])[None, :, None]
    live = torch.ones(B, T, dtype=torch.bool, device=dev)
    if "lens" in s:
        live = torch.arange(T, device=dev)[None] < s["lens"][:, None]
    keep = torch.where(live[:, None], alpha, 1.0)[..., None, None]
    mask = live[:, None, :, None]
    scale = s["attn_scale"]
    q, k, v = torch.where(mask, q, 0.0), torch.where(mask, k, 0.0), torch.where(mask, v, 0.0)
    S = s["S0"].clone() if "S0" in s else torch.zeros(B, H, case["dv"], case["dk"], dtype=torch.float64, device=dev)
    out = torch.zeros_like(v)
    bwd = case["op"] == "lin_bwd"
    if bwd:
        do = torch.where(mask, s["dO"], 0.0) * scale
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(T):
        S = torch.baddbmm((keep[:, :, t] * S).flatten(0, 1), v[:, :, t].flatten(0, 1)[:, :, None],
                          k[:, :, t].flatten(0, 1)[:, None, :]).unflatten(0, (B, H))
        if bwd:
            dq[:, :, t] = (do[:, :, t, None, :] @ S)[:, :, 0]
        else:
            out[:, :, t] = scale * (S @ q[:, :, t, :, None])[..., 0]
    if not bwd:
        return {"O": out[:, :, 0] if step else out, "S": S}
    D = s["dS"].clone() if "dS" in s else torch.zeros_like(S)
    share = (D * S).sum((-1, -2))
    dla = torch.zeros(B, H, T, dtype=torch.float64, device=dev)
    for t in reversed(range(T)):
        D = torch.baddbmm(D.flatten(0, 1), do[:, :, t].flatten(0, 1)[:, :, None],
                          q[:, :, t].flatten(0, 1)[:, None, :]).unflatten(0, (B, H))
        dk[:, :, t] = (v[:, :, t, None, :] @ D)[:, :, 0]
        dv[:, :, t] = (D @ k[:, :, t, :, None])[..., 0]
        # <D_t, S_t> gains what the token read and loses what it wrote
        share = share + (q[:, :, t] * dq[:, :, t]).sum(-1) - (k[:, :, t] * dk[:, :, t]).sum(-1)
        dla[:, :, t] = share
        D = keep[:, :, t] * D
    zero = lambda x: torch.where(mask, x, 0.0)  # noqa: E731
    grads = {"dv": zero(dv), "dq": zero(dq).reshape(B, case["Hq"], -1, T, case["dk"]).sum(2),
             "dk": zero(dk).reshape(B, case["Hk"], -1, T, case["dk"]).sum(2)}
    dla = torch.where(live[:, None], dla, 0.0)
    if case["decay"] == "head":
        grads["dlog_alpha"] = dla.sum((0, 2))
    elif case["decay"] == "token":
        grads["dlog_alpha"] = torch.where(alpha == 0, 0.0, dla)
    if case["state"]:
        grads["dS0"] = D
    return grads


def _exact_block(case, s):
    D, o, x, g = case["D"], s["o"], s["x"], s["gate"]
    one = torch.ones(D, dtype=torch.float64, device=o.device)
    scale = s["scale"] if s["scale"] is not None else one
    w = s["w_post"] if case["post"] else one
    std = ((o ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() if case["post"] else torch.ones_like(o[..., :1])
    if g is None:
        act, slope = torch.ones_like(o), None
    elif case["gate"] == "sigmoid":
        act, slope = torch.sigmoid(g), torch.sigmoid(g) * torch.sigmoid(-g)
    else:
        act, slope = g * torch.sigmoid(g), torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    n = o / std
    if case["op"] == "block_fwd":
        x = x + scale * act * n * w
        return {"x": x, "y": x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * s["w_pre"]}
    xstd = ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt()
    p = s["dy"] * s["w_pre"]
    dx = s["dx_out"] + p / xstd - x * (p * x).sum(-1, keepdim=True) / (D * xstd ** 3)
    m = dx * scale * act * w
    do = m / std - o * (m * o).sum(-1, keepdim=True) / (D * std ** 3) if case["post"] else m
    out = {"dx": dx, "dw_pre": (s["dy"] * x / xstd).sum((0, 1)), "do": do}
    if s["scale"] is not None:
        out["dscale"] = (dx * act * n * w).sum((0, 1))
    if slope is not None:
        out["dgate"] = dx * scale * n * w * slope
    if case["post"]:
        out["dw_post"] = (dx * scale * act * n).sum((0, 1))
    return out
