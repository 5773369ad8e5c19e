"""The operators around a recurrent mixing layer: what each computes and how large it is in use.

A layer built on a recurrence (the gated delta rule, or a selective state space) runs a short causal convolution over
its projected inputs, the recurrence, and a normalisation of each head's output with an activation and a gate. Three
operators, each for whole sequences, for single tokens, and with its gradient:

  conv   p_t = bias + sum_j weight_j x_{t-W+1+j} per channel, y = silu(p); the last W-1 inputs are the state
  ssm    h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t per channel and state, y_t = (C_t . h_t + D x_t) silu(z_t), with
         dt = softplus(raw + bias)
  norm   n = (x - mean) / sqrt(var + eps) over each head of each token (mean = 0 where it is not centred),
         y = (n weight + bias) silu(z), or silu(n weight + bias) without a gate

`lens` holds each sequence's length in a batch padded to T rows: outputs and gradients behind it are zero, and the
final state is the state at that length.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    def conv(name, op, **k):
        return {"name": name, "op": op, "dtype": "bf16", "W": 4, "H": 1, "lens": False, "state": False, **k}

    def ssm(name, op, **k):
        return {"name": name, "op": op, "dtype": "bf16", "N": 16, "G": 1, "lens": False, "state": False, **k}

    def norm(name, op, **k):
        return {"name": name, "op": op, "dtype": "bf16", "xdtype": "f32", "center": False, "gate": True, "heads_first": True,
                "shared": True, **k}

    return [
        # values of 16 heads of 128, written head by head as the delta rule reads them
        conv("conv prompts", "conv_fwd", B=4, T=4096, D=2048, H=16),
        # keys of 30 heads of 96, prompts of different lengths that go on from a cached state
        conv("conv ragged f32", "conv_fwd", B=3, T=1021, D=2880, H=30, dtype="f32", lens=True, state=True),
        # one decode step of 64 sequences
        conv("conv token", "conv_step", B=64, T=1, D=2048, state=True),
        # the training step's gradient at the shape of the first case
        conv("conv gradient", "conv_bwd", B=4, T=4096, D=2048, H=16),
        # prompts of a batch through a layer of 2048 channels and 16 states
        ssm("ssm prompts", "ssm_fwd", B=4, T=4096, D=2048),
        # one long prompt through a narrow layer: few channels, so the length has to give the parallel work
        ssm("ssm long", "ssm_fwd", B=1, T=32768, D=1024),
        # odd sizes: padded prompts, three groups of B and C, continued from a state, in 32 bits
        ssm("ssm ragged f32", "ssm_fwd", B=3, T=517, D=717, N=24, G=3, dtype="f32", lens=True, state=True),
        # one decode step of 64 sequences
        ssm("ssm token", "ssm_step", B=64, T=1, D=2048, state=True),
        # the training step's gradient of two sequences
        ssm("ssm gradient", "ssm_bwd", B=2, T=4096, D=2048),
        # a padded batch's gradient in 32 bits, back to the state that it went on from
        ssm("ssm gradient ragged f32", "ssm_bwd", B=2, T=333, D=486, dtype="f32", lens=True, state=True),
        # the delta rule's output [B, heads, T, 128] in 32 bits, normalised and gated into [B, T, heads x 128]
        norm("norm prompts", "norm_fwd", B=4, T=4096, G=16, d=128),
        # its gradient at 30 heads of 192, with a weight for every head and a centred mean
        norm("norm gradient", "norm_bwd", B=2, T=1031, G=30, d=192, xdtype="bf16", center=True, shared=False),
    ]


def _between(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_fwd", "ssm_bwd", "ssm_step", "norm_fwd", "norm_bwd"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    B = _between(rng, 1, 128 if op.endswith("step") else 8)
    T = 1 if op.endswith("step") else _between(rng, 1, 8192)
    if op.startswith("norm"):
        G, d = _between(rng, 1, 32), _between(rng, 8, 512)
        T = max(1, min(T, (32 << 20) // (B * G * d)))
        return {**c, "xdtype": rng.choice(["bf16", "f32"]), "B": B, "T": T, "G": G, "d": d, "center": rng.random() < 0.5,
                "gate": rng.random() < 0.7, "heads_first": rng.random() < 0.5, "shared": rng.random() < 0.5}
    c.update(B=B, T=T, lens=op[-4:] != "step" and rng.random() < 0.5, state=op[-4:] == "step" or rng.random() < 0.5)
    if op.startswith("conv"):
        H = rng.choice([1, 1, 8, 30])
        hd = max(1, _between(rng, 16, 4096) // H)
        c.update(W=rng.choice([2, 3, 4, 4]), H=1 if op == "conv_step" else H, D=H * hd)
        c["T"] = max(1, min(T, (32 << 20) // (B * H * hd)))
        return c
    N, G = rng.choice([1, 4, 7, 8, 16, 16, 16, 24, 32, 64]), rng.choice([1, 1, 1, 2, 3])
    D = G * max(1, _between(rng, 16, 4096) // G)
    return {**c, "N": N, "G": G, "D": D, "T": max(1, min(T, (1 << 28) // (B * D * N)))}


def prepare(case, seed):
    op, dev = case["op"], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, T, dt = case["B"], case["T"], DTYPES[case["dtype"]]

    def rnd(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"op": op, "case": dict(case)}
    if case.get("lens"):
        # different lengths, one sequence that fills its row
        lens = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        lens[0] = T
        s["lens"] = lens
    if op.startswith("conv"):
        D, W, H = case["D"], case["W"], case["H"]
        # the inputs are a slice of a wider projection's output
        s["x"] = rnd(B, T, D + 64, dtype=dt)[:, :, 32:32 + D]
        s["weight"] = rnd(D, W, std=W ** -0.5)
        s["bias"] = rnd(D, std=0.1)
        if case["state"]:
            s["state0"] = rnd(B, W - 1, D, dtype=dt)
        if op == "conv_bwd":
            s["dy"] = rnd(B, H, T, D // H, dtype=dt)
            if case["state"]:
                s["dstate"] = rnd(B, W - 1, D, dtype=dt)
        if op == "conv_step":
            s["x"] = s["x"][:, 0]
        return s
    if op.startswith("ssm"):
        D, N, G = case["D"], case["N"], case["G"]
        s["x"] = torch.nn.functional.silu(rnd(B, T, D)).to(dt)
        # B and C are slices of one projection's output, z of another's
        bc = rnd(B, T, 2 * G * N + 16, dtype=dt)
        s["Bm"] = bc[:, :, 16:16 + G * N].unflatten(2, (G, N))
        s["C"] = bc[:, :, 16 + G * N:].unflatten(2, (G, N))
        s["z"] = rnd(B, T, 2 * D, dtype=dt)[:, :, D:]
        s["dt"] = rnd(B, T, D, std=0.5, dtype=dt)
        # step sizes from 1e-3 to 1e-1, decay rates near 1, 2, ..., N
        step = torch.exp(torch.rand(D, generator=g, device=dev) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(rnd(D, N, std=0.2))
        s["D"] = 1.0 + rnd(D, std=0.1)
        if case["state"]:
            s["h0"] = rnd(B, D, N, std=0.3)
        if op == "ssm_bwd":
            s["dy"] = rnd(B, T, D, dtype=dt)
            if case["state"]:
                s["dh"] = rnd(B, D, N, std=0.3)
        if op == "ssm_step":
            for k in ("x", "dt", "Bm", "C", "z"):
                s[k] = s[k][:, 0]
        return s
    G, d, xdt = case["G"], case["d"], DTYPES[case["xdtype"]]
    s["x"] = rnd(B, G, T, d, dtype=xdt).transpose(1, 2) if case["heads_first"] else rnd(B, T, G, d, dtype=xdt)
    wshape = (d,) if case["shared"] else (G, d)
    s["weight"] = 1.0 + rnd(*wshape, std=0.1)
    s["bias"] = rnd(*wshape, std=0.1) if case["center"] else None
    s["z"] = rnd(B, T, G, d, dtype=dt) if case["gate"] else None
    if op == "norm_bwd":
        s["dy"] = rnd(B, T, G, d, dtype=dt)
    return s


def run(s):
    if own:
        return _own(s)
    return {"conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd, "conv_step": _conv_step, "ssm_fwd": _ssm_fwd, "ssm_bwd": _ssm_bwd,
            "ssm_step": _ssm_step, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}[s["op"]](s)


def _own(s):
    import gated_delta_rule_13_amd as gdn
    op, c = s["op"], s["case"]
    if op == "conv_fwd":
        y, state = gdn.gdn_conv_fwd(s["x"], s["weight"], s["bias"], s.get("state0"), lens=s.get("lens"), heads=c["H"])
        return {"y": y, "state": state}
    if op == "conv_bwd":
        return gdn.gdn_conv_bwd(s["dy"], s["x"], s["weight"], s["bias"], s.get("state0"), lens=s.get("lens"),
                                dstate_out=s.get("dstate"))
    if op == "conv_step":
        return {"y": gdn.gdn_conv_step(s["x"], s["weight"], s["bias"], s["state0"]), "state": s["state0"]}
    if op == "ssm_fwd":
        y, h = gdn.gdn_ssm_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["C"], s["D"], s["z"], s["dt_bias"], s.get("h0"),
                               lens=s.get("lens"))
        return {"y": y, "h": h}
    if op == "ssm_bwd":
        return gdn.gdn_ssm_bwd(s["dy"], s["x"], s["dt"], s["A"], s["Bm"], s["C"], s["D"], s["z"], s["dt_bias"], s.get("h0"),
                               lens=s.get("lens"), dh_final=s.get("dh"))
    if op == "ssm_step":
        return {"y": gdn.gdn_ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["C"], s["D"], s["z"], s["dt_bias"], h=s["h0"]),
                "h": s["h0"]}
    if op == "norm_fwd":
        return {"y": gdn.gdn_norm_fwd(s["x"], s["weight"], s["bias"], s["z"], center=c["center"], eps=EPS,
                                      o_dtype=DTYPES[c["dtype"]])}
    return gdn.gdn_norm_bwd(s["dy"], s["x"], s["weight"], s["bias"], s["z"], center=c["center"], eps=EPS)


def _inside(s):
    """[B, T, 1]: whether a row belongs to its sequence."""
    B, T = s["x"].shape[:2]
    if "lens" not in s:
        return torch.ones(B, T, 1, dtype=torch.bool, device=s["x"].device)
    return (torch.arange(T, device=s["x"].device)[None, :] < s["lens"][:, None])[:, :, None]


def _silu_and_slope(p):
    e = 1.0 / (1.0 + torch.exp(-p))
    return p * e, e * (1.0 + p * (1.0 - e))


def _softplus(u):
    return u.clamp(min=0.0) + torch.log1p(torch.exp(-u.abs()))


def _conv_pre(s):
    """The state followed by the inputs, its windows [B, T, D, W], and the sums before the activation, in 32 bits."""
    x = s["x"].float()
    B, T, D = x.shape
    W = s["weight"].shape[1]
    past = s["state0"].float() if "state0" in s else x.new_zeros(B, W - 1, D)
    rows = torch.cat([past, x], 1)
    win = rows.unfold(1, W, 1)
    return rows, win, s["bias"] + (win * s["weight"]).sum(-1)


def _tail(s, rows):
    """The W-1 rows that end at each sequence's length, and their places."""
    B, T, D = s["x"].shape
    W = s["weight"].shape[1]
    n = s["lens"].long() if "lens" in s else torch.full((B,), T, device=rows.device)
    at = (n[:, None] + torch.arange(W - 1, device=rows.device))[:, :, None].expand(B, W - 1, D)
    return rows.gather(1, at), at


def _conv_fwd(s):
    rows, _, p = _conv_pre(s)
    B, T, D = s["x"].shape
    H = s["case"]["H"]
    y = torch.where(_inside(s), _silu_and_slope(p)[0], 0.0).to(s["x"].dtype)
    return {"y": y.unflatten(2, (H, D // H)).transpose(1, 2).contiguous(), "state": _tail(s, rows)[0].to(s["x"].dtype)}


def _conv_bwd(s):
    rows, win, p = _conv_pre(s)
    B, T, D = s["x"].shape
    w = s["weight"]
    W = w.shape[1]
    dy = s["dy"].float().transpose(1, 2).reshape(B, T, D)
    dp = torch.where(_inside(s), dy * _silu_and_slope(p)[1], 0.0)
    out = {"dweight": (dp[:, :, :, None] * win).sum((0, 1)), "dbias": dp.sum((0, 1))}
    # row r of the state and inputs meets the taps of rows r-W+1 .. r of the outputs
    after = torch.cat([dp.new_zeros(B, W - 1, D), dp, dp.new_zeros(B, W - 1, D)], 1).unfold(1, W, 1)
    drows = (after * w.flip(1)).sum(-1)
    if "dstate" in s:
        drows = drows.scatter_add(1, _tail(s, rows)[1], s["dstate"].float())
    out["dx"] = drows[:, W - 1:].to(s["x"].dtype)
    if "state0" in s:
        out["dstate0"] = drows[:, :W - 1].to(s["x"].dtype)
    return out


def _conv_step(s):
    win = torch.cat([s["state0"], s["x"][:, None]], 1)
    p = s["bias"] + (win.float() * s["weight"].t()).sum(1)
    s["state0"].copy_(win[:, 1:])
    return {"y": _silu_and_slope(p)[0].to(s["x"].dtype), "state": s["state0"]}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along dimension 1, by doubling the span that each row covers."""
    k, T = 1, a.shape[1]
    while k < T:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1) if 2 * k < T else a
        k *= 2
    return b


def _by_channel(m, D):
    """[.., G, N] -> [.., D, N]: each group's row for all its channels."""
    return m.float().repeat_interleave(D // m.shape[-2], dim=-2)


def _ssm_parts(s):
    """The step sizes, decays and states, with rows behind a sequence's end leaving the state as it is."""
    ins = _inside(s)
    x, D = s["x"].float(), s["x"].shape[2]
    u = s["dt"].float() + s["dt_bias"]
    dt = torch.where(ins, _softplus(u), 0.0)
    x = torch.where(ins, x, 0.0)
    Bm, C = _by_channel(s["Bm"], D), _by_channel(s["C"], D)
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * Bm
    if "h0" in s:
        b[:, 0] += a[:, 0] * s["h0"]
    return ins, x, u, dt, Bm, C, a, _scan(a, b)


def _ssm_fwd(s):
    ins, x, _, _, _, C, _, h = _ssm_parts(s)
    y = (h * C).sum(-1) + s["D"] * x
    y = torch.where(ins, y * _silu_and_slope(s["z"].float())[0], 0.0)
    return {"y": y.to(s["x"].dtype), "h": h[:, -1].contiguous()}


def _ssm_bwd(s):
    ins, x, u, dt, Bm, C, a, h = _ssm_parts(s)
    B, T, D = x.shape
    G, N = s["Bm"].shape[2:]
    io = s["x"].dtype
    gate, slope = _silu_and_slope(s["z"].float())
    dy = torch.where(ins, s["dy"].float(), 0.0)
    dz = dy * slope * ((h * C).sum(-1) + s["D"] * x)
    dy = dy * gate
    # gh_t = C_t dy_t + a_{t+1} gh_{t+1}
    gh = dy[..., None] * C
    if "dh" in s:
        gh[:, -1] += s["dh"]
    decay = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    gh = _scan(decay.flip(1), gh.flip(1)).flip(1)
    past = torch.cat([s["h0"][:, None] if "h0" in s else torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    du = (gh * Bm).sum(-1)
    da = gh * past * a
    draw_raw = torch.where(ins, (x * du + (da * s["A"]).sum(-1)) / (1.0 + torch.exp(-u)), 0.0)
    out = {"dx": torch.where(ins, s["D"] * dy + dt * du, 0.0).to(io), "ddt": draw_raw.to(io), "dz": dz.to(io),
           "dA": (da * dt[..., None]).sum((0, 1)), "dD": (dy * x).sum((0, 1)), "ddt_bias": draw_raw.sum((0, 1)),
           "dB": (gh * (dt * x)[..., None]).unflatten(2, (G, D // G)).sum(3).to(io),
           "dC": (h * dy[..., None]).unflatten(2, (G, D // G)).sum(3).to(io)}
    if "h0" in s:
        out["dh0"] = (a[:, 0] * gh[:, 0]).contiguous()
    return out


def _ssm_step(s):
    x, D = s["x"].float(), s["x"].shape[1]
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(dt[..., None] * s["A"]) * s["h0"] + (dt * x)[..., None] * _by_channel(s["Bm"], D)
    y = (h * _by_channel(s["C"], D)).sum(-1) + s["D"] * x
    s["h0"].copy_(h)
    return {"y": (y * _silu_and_slope(s["z"].float())[0]).to(s["x"].dtype), "h": s["h0"]}


def _norm_parts(s):
    x = s["x"].float()
    if s["case"]["center"]:
        x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    p = n * s["weight"]
    return r, n, p + s["bias"] if s["bias"] is not None else p


def _norm_fwd(s):
    _, _, p = _norm_parts(s)
    y = p * _silu_and_slope(s["z"].float())[0] if s["z"] is not None else _silu_and_slope(p)[0]
    return {"y": y.to(DTYPES[s["case"]["dtype"]])}


def _norm_bwd(s):
    r, n, p = _norm_parts(s)
    dy, out = s["dy"].float(), {}
    if s["z"] is not None:
        gate, slope = _silu_and_slope(s["z"].float())
        out["dz"] = (dy * p * slope).to(s["z"].dtype)
        dp = dy * gate
    else:
        dp = dy * _silu_and_slope(p)[1]
    over = (0, 1, 2) if s["case"]["shared"] else (0, 1)
    out["dweight"] = (dp * n).sum(over)
    if s["bias"] is not None:
        out["dbias"] = dp.sum(over)
    dn = dp * s["weight"]
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if s["case"]["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    out["dx"] = (r * dx).to(s["x"].dtype)
    return out


def work(case):
    op, B, T = case["op"], case["B"], case["T"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        n, xe = B * T * case["G"] * case["d"], 2 if case["xdtype"] == "bf16" else 4
        gate = e if case["gate"] else 0
        if op == "norm_fwd":
            return {"bytes": n * (xe + e + gate), "flops": n * 10}
        return {"bytes": n * (2 * xe + e + 2 * gate), "flops": n * 25}
    D = case["D"]
    n = B * T * D
    if op.startswith("conv"):
        W = case["W"]
        state = B * (W - 1) * D * e
        if op == "conv_bwd":
            return {"bytes": 3 * n * e + (3 * state if case["state"] else 0) + 4 * D * (W + 1) * 2, "flops": n * (6 * W + 10)}
        return {"bytes": 2 * n * e + state * (2 if case["state"] else 1) + 4 * D * (W + 1), "flops": n * (2 * W + 5)}
    N, G = case["N"], case["G"]
    state, bc, par = B * D * N * 4, 2 * B * T * G * N * e, 4 * D * (N + 2)
    if op == "ssm_bwd":
        # x, dt, z, dy read, dx, ddt, dz written
        return {"bytes": 7 * n * e + 2 * bc + 2 * par + (3 * state if case["state"] else 0), "flops": n * (20 * N + 30)}
    return {"bytes": 4 * n * e + bc + par + state * (2 if case["state"] else 1), "flops": n * (6 * N + 20)}


def exact(case, seed):
    """The operators from their definitions in 64 bits, a token at a time where they are recurrences."""
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    op, B, T = case["op"], case["B"], case["T"]
    sig = torch.sigmoid
    if op.startswith("norm"):
        return _exact_norm(case, s, sig)
    one = op.endswith("step")
    if one:
        s.update({k: s[k][:, None] for k in ("x", "dt", "Bm", "C", "z") if k in s})
    x = s["x"]
    D = x.shape[2]
    lens = s["lens"].tolist() if "lens" in s else [T] * B
    return (_exact_conv if op.startswith("conv") else _exact_ssm)(case, s, sig, x, lens, one, B, T, D)


def _exact_norm(case, s, sig):
    x, w, b, z, d = s["x"], s["weight"], s["bias"], s["z"], case["d"]
    mean = x.sum(-1, keepdim=True) / d if case["center"] else torch.zeros_like(x[..., :1])
    std = (((x - mean) ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
    n = (x - mean) / std
    p = n * w + (b if b is not None else 0.0)
    at = z if z is not None else p
    silu, slope = at * sig(at), sig(at) + at * sig(at) * sig(-at)
    if case["op"] == "norm_fwd":
        return {"y": p * silu if z is not None else silu}
    dy = s["dy"]
    dp = dy * (silu if z is not None else slope)
    over = (0, 1, 2) if case["shared"] else (0, 1)
    dn = dp * w
    dx = dn / std - n * (dn * n).sum(-1, keepdim=True) / (d * std)
    if case["center"]:
        dx = dx - dn.sum(-1, keepdim=True) / (d * std)
    return {"dx": dx, "dweight": (dp * n).sum(over), **({"dbias": dp.sum(over)} if b is not None else {}),
            **({"dz": dy * p * slope} if z is not None else {})}


def _exact_conv(case, s, sig, x, lens, one, B, T, D):
    W, H, w = case["W"], case["H"], s["weight"]
    past = s["state0"] if "state0" in s else x.new_zeros(B, W - 1, D)
    rows = torch.cat([past, x], 1)
    p = s["bias"].expand(B, T, D).clone()
    for j in range(W):
        p += w[:, j] * rows[:, j:j + T]
    state = torch.stack([rows[b, n:n + W - 1] for b, n in enumerate(lens)])
    if case["op"] != "conv_bwd":
        y = p * sig(p)
        for b, n in enumerate(lens):
            y[b, n:] = 0
        if one:
            return {"y": y[:, 0], "state": state}
        return {"y": y.reshape(B, T, H, D // H).permute(0, 2, 1, 3).contiguous(), "state": state}
    dp = s["dy"].permute(0, 2, 1, 3).reshape(B, T, D) * (sig(p) + p * sig(p) * sig(-p))
    for b, n in enumerate(lens):
        dp[b, n:] = 0
    drows, dw = torch.zeros_like(rows), torch.zeros_like(w)
    for j in range(W):
        drows[:, j:j + T] += w[:, j] * dp
        dw[:, j] = (dp * rows[:, j:j + T]).sum((0, 1))
    if "dstate" in s:
        for b, n in enumerate(lens):
            drows[b, n:n + W - 1] += s["dstate"][b]
    return {"dx": drows[:, W - 1:], "dweight": dw, "dbias": dp.sum((0, 1)), **({"dstate0": drows[:, :W - 1]} if "state0" in s else {})}


def _exact_ssm(case, s, sig, x, lens, one, B, T, D):
    N, G, A, z = case["N"], case["G"], s["A"], s["z"]
    if case["op"] == "ssm_bwd" and B * T * D * N > 1 << 29:
        return None
    u = s["dt"] + s["dt_bias"]
    dt = torch.logaddexp(u, torch.zeros_like(u))
    live = torch.arange(T, device=x.device)[None, :] < torch.tensor(lens, device=x.device)[:, None]
    wide = lambda m, t: m[:, t].repeat_interleave(D // G, dim=1)  # noqa: E731
    h = s["h0"].clone() if "h0" in s else x.new_zeros(B, D, N)
    keep, scan = [h], torch.zeros_like(x)
    for t in range(T):
        new = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * wide(s["Bm"], t)
        h = torch.where(live[:, t, None, None], new, h)
        scan[:, t] = (h * wide(s["C"], t)).sum(-1)
        if case["op"] == "ssm_bwd":
            keep.append(h)
    scan = scan + s["D"] * x
    mask = live[:, :, None]
    if case["op"] != "ssm_bwd":
        y = torch.where(mask, scan * z * sig(z), 0.0)
        return {"y": y[:, 0] if one else y, "h": h}
    dy = torch.where(mask, s["dy"], 0.0)
    dz = dy * scan * (sig(z) + z * sig(z) * sig(-z))
    dy = dy * z * sig(z)
    gh = s["dh"].clone() if "dh" in s else torch.zeros_like(h)
    dx, ddt, dA = s["D"] * dy, torch.zeros_like(x), torch.zeros_like(A)
    dB, dC = torch.zeros_like(s["Bm"]), torch.zeros_like(s["C"])
    for t in reversed(range(T)):
        on = live[:, t, None, None]
        step, a = dt[:, t, :, None], torch.exp(dt[:, t, :, None] * A)
        full = gh + dy[:, t, :, None] * wide(s["C"], t)
        through = torch.where(on, full, 0.0)
        du = (through * wide(s["Bm"], t)).sum(-1)
        da = through * keep[t] * a
        dx[:, t] += dt[:, t] * du
        ddt[:, t] = x[:, t] * du + (da * A).sum(-1)
        dA += (da * step).sum(0)
        dB[:, t] = (through * step * x[:, t, :, None]).reshape(B, G, D // G, N).sum(2)
        dC[:, t] = torch.where(on, keep[t + 1] * dy[:, t, :, None], 0.0).reshape(B, G, D // G, N).sum(2)
        gh = torch.where(on, a * full, gh)
    ddt = torch.where(mask, ddt * sig(u), 0.0)
    return {"dx": torch.where(mask, dx, 0.0), "ddt": ddt, "dz": dz, "dA": dA, "dB": dB, "dC": dC, "dD": (dy * torch.where(mask, x, 0.0)).sum((0, 1)),
            "ddt_bias": ddt.sum((0, 1)), **({"dh0": gh} if "h0" in s else {})}
