"""The operators around the recurrence in 64 bits, a token at a time, and the
comparison of a kernel's outputs with them.

Plain torch on float64 tensors, differentiable: gradients of the references
come from torch's autograd, and from central differences of them.

Tolerance.  A number that a kernel returns is off by the rounding to its own
type (half a step: ``torch.finfo(t).eps / 2``, relative to it) and by the fp32
arithmetic before it.  There every factor of a product carries a bounded
number of roundings u = 2^-24: a step size (softplus) about 12, a decay
exp(s A) with |s A| <= 8 about 8 (12 + 2) + 2 = 114 at most, an activation
about 8.  A state weighs that error by the decay itself (what is far below 1
is forgotten), so that |s A| exp(-|s A|) <= 1/e bounds what a step adds, about
6 u, over a memory of at most 1 / (1 - exp(-|s A|)) steps, whose errors are
independent roundings.  Sums of mixed signs keep their absolute errors.  160 u
= 1e-5 of a tensor's largest number covers these chains; it is also the bound
that the chunked kernels are held to for fp32.
"""
from __future__ import annotations

import torch

FP32_TOL = 1e-5


def close(name, got, want, scale=None):
    """got (a kernel's output) against want (fp64): every number within half a
    step of its type of the exact one, plus FP32_TOL of the tensor's largest
    (or of `scale`)."""
    assert tuple(got.shape) == tuple(want.shape), (name, tuple(got.shape), tuple(want.shape))
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    if w.numel() == 0:
        return
    assert torch.isfinite(g).all(), f"{name}: numbers that are not finite"
    top = float(w.abs().max()) if scale is None else scale
    off = (g - w).abs() - torch.finfo(got.dtype).eps / 2 * w.abs() - FP32_TOL * top
    worst = float(off.max())
    assert worst <= 0, f"{name}: off by {worst:.3e} more than allowed (largest number {top:.3e})"


def live_rows(B, T, lens):
    """[B, T] bool: the rows that belong to their sequence."""
    if lens is None:
        return torch.ones(B, T, dtype=torch.bool)
    return torch.arange(T)[None] < lens.cpu().clamp(0, T)[:, None]


def silu(x):
    return x / (1 + torch.exp(-x))


def conv(x, weight, bias=None, state0=None, lens=None, heads=None, act="silu"):
    """-> y, state_out"""
    B, T, D = x.shape
    W = weight.shape[1]
    live = live_rows(B, T, lens)
    x = torch.where(live[:, :, None], x, torch.zeros((), dtype=x.dtype))
    past = torch.zeros(B, W - 1, D, dtype=x.dtype) if state0 is None else state0
    rows = torch.cat([past, x], 1)
    ys = []
    for t in range(T):
        p = (rows[:, t:t + W] * weight.t()).sum(1)
        if bias is not None:
            p = p + bias
        ys.append(silu(p) if act == "silu" else p)
    y = torch.where(live[:, :, None], torch.stack(ys, 1), torch.zeros((), dtype=x.dtype))
    n = [T] * B if lens is None else lens.cpu().clamp(0, T).tolist()
    state = torch.stack([rows[b, n[b]:n[b] + W - 1] for b in range(B)])
    if heads is not None:
        y = y.reshape(B, T, heads, D // heads).transpose(1, 2)
    return y, state


def ssm(x, dt, A, Bm, C, D=None, z=None, dt_bias=None, h0=None, lens=None, dt_softplus=True):
    """-> y, h_final"""
    B, T, Dc = x.shape
    G, N = Bm.shape[2:]
    live = live_rows(B, T, lens)
    zero = torch.zeros((), dtype=x.dtype)
    # (rows behind a length are taken out before anything is computed from
    # them, so that autograd multiplies nothing by their NaN)
    dt, x = (torch.where(live[:, :, None], v, zero) for v in (dt, x))
    s = dt if dt_bias is None else dt + dt_bias
    if dt_softplus:
        s = torch.logaddexp(s, zero)
    s = torch.where(live[:, :, None], s, zero)
    Bm, C = (torch.where(live[:, :, None, None], v, zero).repeat_interleave(Dc // G, dim=2) for v in (Bm, C))
    h = torch.zeros(B, Dc, N, dtype=x.dtype) if h0 is None else h0
    ys = []
    for t in range(T):
        h = torch.exp(s[:, t, :, None] * A) * h + (s[:, t] * x[:, t])[..., None] * Bm[:, t]
        ys.append((h * C[:, t]).sum(-1))
    y = torch.stack(ys, 1)
    if D is not None:
        y = y + D * x
    if z is not None:
        y = y * silu(torch.where(live[:, :, None], z, zero))
    return torch.where(live[:, :, None], y, zero), h


def norm(x, weight=None, bias=None, z=None, act="silu", center=False, eps=1e-5):
    """-> y"""
    f = silu if act == "silu" else (lambda v: v)
    c = x - x.mean(-1, keepdim=True) if center else x
    p = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    if weight is not None:
        p = p * weight
    if bias is not None:
        p = p + bias
    return p * f(z) if z is not None else f(p)


def wide(args):
    """float64 CPU copies of a dict's floating tensors (exact), the rest as it is."""
    return {k: v.detach().double().cpu() if torch.is_tensor(v) and v.is_floating_point() else v
            for k, v in args.items()}


def gradients(fn, args, names, cotangents):
    """Autograd's gradients of the fp64 reference fn(**args), whose outputs
    have the given cotangents (None: none), for the named arguments."""
    leaves = {n: args[n].clone().requires_grad_(True) for n in names}
    out = fn(**{**args, **leaves})
    out = out if isinstance(out, tuple) else (out,)
    loss = sum((o * c.double().cpu()).sum() for o, c in zip(out, cotangents) if c is not None)
    got = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return {n: torch.zeros_like(leaves[n]) if g is None else g for n, g in zip(names, got)}


def difference(fn, args, name, direction, cotangents, step=1e-4):
    """Central difference of the fp64 reference's loss along one direction of
    one argument (error about step^2 of the third derivative)."""
    def loss(s):
        out = fn(**{**args, name: args[name] + s * direction})
        out = out if isinstance(out, tuple) else (out,)
        return float(sum((o * c.double().cpu()).sum() for o, c in zip(out, cotangents) if c is not None))
    return (loss(step) - loss(-step)) / (2 * step)


def rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def dev(args):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in args.items()}
