"""Linear attention with decay and the norms around a block in 64 bits, and the
comparison of a kernel's outputs with them.  Plain torch on float64 tensors, a
token at a time, differentiable.

Tolerance of linear attention.  Each output is a sum of products; the kernels
round factors of them (the state, decayed values, products of rows with their
decay) to two bf16 numbers, 2^-17 relative at most, and add in fp32, where 2^-24
for each of some 200 terms of one sign is 2^-16.4 at most and less for mixed
signs.  So the error of an element is below 2^-16 of the same sum over absolute
values, which the reference gives on absolute inputs (everything but the signs is
products and sums).  The decay's gradient is in addition a sum over later tokens
of rounded parts q . dq and k . dk, whose errors are independent: 2^-16 times the
root of their number times the largest of them.

Where an output is bf16, the state and the products of rows (not the decayed
values, nor what fp32 outputs and the decay's gradient are made of) are rounded to
one bf16 number: every term of the sum, which holds one of the two, is off by half
a step more, 2^-8 of it.
"""
from __future__ import annotations

import torch

from tests import layer_ref as ref

LIN_TOL = 2.0 ** -16


def lin(q, k, v, log_alpha=None, S0=None, lens=None, scale=1.0):
    """-> O, S_final"""
    B, H, T, dv = v.shape
    live = ref.live_rows(B, T, lens)[:, None, :, None]
    zero = torch.zeros((), dtype=v.dtype)
    q, k, v = (torch.where(live, x.repeat_interleave(H // x.shape[1], 1), zero) for x in (q, k, v))
    if log_alpha is None:
        a = torch.ones(B, H, T, dtype=v.dtype)
    else:
        la = log_alpha if log_alpha.dim() == 3 else log_alpha[None, :, None].expand(B, H, T)
        a = torch.exp(torch.where(live[..., 0], la, zero))
    S = torch.zeros(B, H, dv, q.shape[-1], dtype=v.dtype) if S0 is None else S0
    out = []
    for t in range(T):
        S = a[:, :, t, None, None] * S + v[:, :, t, :, None] * k[:, :, t, None, :]
        out.append(scale * (S @ q[:, :, t, :, None])[..., 0])
    return torch.where(live, torch.stack(out, 2), zero), S


def lin_bound(a, **k):
    """The sums of lin over absolute values."""
    return lin(**{n: x if n in ("log_alpha", "lens") or x is None else x.abs() for n, x in a.items()}, **k)


def within(name, got, want, bound):
    """Every number within half a step of its type of the exact one, plus
    LIN_TOL times `bound` there (bf16: and half a step of the terms)."""
    assert tuple(got.shape) == tuple(want.shape), (name, tuple(got.shape), tuple(want.shape))
    g, w = got.detach().double().cpu(), want.detach().double()
    assert torch.isfinite(g).all(), f"{name}: numbers that are not finite"
    half = torch.finfo(got.dtype).eps / 2
    each = LIN_TOL + (half if got.dtype is torch.bfloat16 else 0)
    off = (g - w).abs() - half * w.abs() - each * bound.detach() * (1 + 2 * half)
    worst = float(off.max())
    assert worst <= 1e-30, f"{name}: off by {worst:.3e} more than allowed (largest number {float(w.abs().max()):.3e})"


def block(o, x, w_pre=None, w_post=None, gate=None, scale=None, act="sigmoid", post=True, eps=1e-5):
    """-> x_out, y"""
    n = o
    if post:
        n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + eps)
        if w_post is not None:
            n = n * w_post
    if gate is not None:
        n = n * (torch.sigmoid(gate) if act == "sigmoid" else ref.silu(gate) if act == "silu" else gate)
    if scale is not None:
        n = n * scale
    x = x + n
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x, y if w_pre is None else y * w_pre
