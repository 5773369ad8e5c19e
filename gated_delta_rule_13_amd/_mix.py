"""Binding of linear attention with decay and of the norms around a block
(``include/gdn.h``).  Argument checks and marshalling only, in the manner of the
operators around the recurrence (``_layer.py``): strided inputs may be views
whose last dimension is contiguous, outputs carry no autograd history, calls run
on ``stream`` (the current stream of the tensors' device by default),
asynchronously.
"""
from __future__ import annotations

import ctypes

import torch

from . import _layer as base
from ._lib import GdnBlockNormShape, GdnLinShape, check, load

__all__ = ["gdn_lin_fwd", "gdn_lin_bwd", "gdn_lin_step", "gdn_lin_fwd_workspace_bytes", "gdn_lin_bwd_workspace_bytes",
           "gdn_block_norm_fwd", "gdn_block_norm_bwd", "gdn_block_norm_bwd_workspace_bytes"]

_F32 = torch.float32
_ACTS = {None: 0, "sigmoid": 1, "silu": 2}


# ---- linear attention ----

def _lin_shape(q, k, v, log_alpha, scale, o_dtype):
    """The shape structure of q [B,Hq,T,d_k], k, v, checked but for devices."""
    base._rank("q", q, 4)
    base._rank("k", k, 4)
    base._rank("v", v, 4)
    B, H, T, dv = v.shape
    Hq, Hk, dk = q.shape[1], k.shape[1], q.shape[3]
    if Hq < 1 or Hk < 1 or H % Hq or H % Hk:
        raise ValueError(f"{H} heads of values do not divide among {Hq} of queries and {Hk} of keys")
    per_head, a = 0, (0, 0, 0)
    if log_alpha is not None:
        if log_alpha.dim() == 1:
            per_head = 1
        else:
            base._rank("log_alpha", log_alpha, 3)
            a = log_alpha.stride()
    return GdnLinShape(B, H, T, Hq, Hk, dk, dv, base._code(v.dtype), base._code(o_dtype), per_head, float(scale),
                       *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *a)


def _lin_check(s, q, k, v, log_alpha, S0, lens, dev):
    io = v.dtype
    base._check("q", q, (s.B, s.Hq, s.T, s.d_k), io, dev, 1)
    base._check("k", k, (s.B, s.Hk, s.T, s.d_k), io, dev, 1)
    base._check("v", v, (s.B, s.H, s.T, s.d_v), io, dev, 1)
    _check_decay(log_alpha, s.H, (s.B, s.H, s.T), dev)
    base._check("S0", S0, (s.B, s.H, s.d_v, s.d_k), _F32, dev)
    base._check("lens", lens, (s.B,), torch.int32, dev)


def _check_decay(log_alpha, H, full, dev):
    """log_alpha [H], contiguous, or of the full shape with any strides."""
    if log_alpha is None:
        return
    if log_alpha.dim() == 1:
        base._check("log_alpha", log_alpha, (H,), _F32, dev)
        return
    if log_alpha.shape != full:
        raise ValueError(f"log_alpha must have shape {tuple(full)} or ({H},), got {tuple(log_alpha.shape)}")
    if log_alpha.dtype is not _F32:
        raise TypeError(f"log_alpha must be {_F32}, got {log_alpha.dtype}")
    if log_alpha.device != dev:
        raise ValueError(f"log_alpha must be on {dev}, got {log_alpha.device}")


def gdn_lin_fwd_workspace_bytes(shape: GdnLinShape) -> int:
    return base._query("gdn_lin_fwd_workspace_bytes", shape)


def gdn_lin_fwd(q, k, v, log_alpha=None, S0=None, lens=None, scale=1.0, o_dtype=None, O=None, S_final=None, stream=None):
    """Linear attention with a decay for each head:
        S_t = exp(log_alpha_t) S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t.
    q [B,Hq,T,d_k], k [B,Hk,T,d_k], v [B,H,T,d_v] of one dtype, bf16 or fp32,
    views with a contiguous last dimension (d_k, d_v <= 256); H is a multiple of
    Hq and Hk, head h of v reads heads h // (H // Hq) and h // (H // Hk).
    log_alpha fp32 [B,H,T], a view with any strides, or [H], or None (no decay);
    -inf starts anew at its token.  S0 [B,H,d_v,d_k] fp32 or None (zero); lens [B]
    int32 or None, the tokens of each sequence in a padded batch (rows behind are
    written as zero).  Returns (O [B,H,T,d_v] in o_dtype (default: v's),
    S_final [B,H,d_v,d_k] fp32), which may be passed in; S_final may be S0."""
    if base._elsewhere(v, stream):
        with base._moved("gdn_lin_fwd", v, stream):
            return gdn_lin_fwd(q, k, v, log_alpha, S0, lens, scale, o_dtype, O, S_final)
    dev = v.device
    if o_dtype is None:
        o_dtype = v.dtype if O is None else O.dtype
    s = _lin_shape(q, k, v, log_alpha, scale, o_dtype)
    _lin_check(s, q, k, v, log_alpha, S0, lens, dev)
    if O is None:
        O = torch.empty((s.B, s.H, s.T, s.d_v), dtype=o_dtype, device=dev)
    else:
        base._check("O", O, (s.B, s.H, s.T, s.d_v), o_dtype, dev)
        base._separate("O", O, q=q, k=k, v=v, log_alpha=log_alpha, S0=S0, lens=lens)
    if S_final is None:
        S_final = torch.empty((s.B, s.H, s.d_v, s.d_k), dtype=_F32, device=dev)
    else:
        base._check("S_final", S_final, (s.B, s.H, s.d_v, s.d_k), _F32, dev)
        same = S0 is not None and S_final.data_ptr() == S0.data_ptr()
        base._separate("S_final", S_final, q=q, k=k, v=v, log_alpha=log_alpha, S0=None if same else S0, lens=lens, O=O)
    nbytes = gdn_lin_fwd_workspace_bytes(s)
    wp, ws = base._workspace(nbytes, dev)
    check(load().gdn_lin_fwd(ctypes.byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), base._ptr(log_alpha), base._ptr(S0),
                             base._ptr(lens), O.data_ptr(), S_final.data_ptr(), wp, nbytes, base._stream(v)))
    return O, S_final


def gdn_lin_step(q, k, v, log_alpha=None, S=None, scale=1.0, o_dtype=None, O=None, stream=None):
    """One token of every sequence: q [B,Hq,d_k], k [B,Hk,d_k], v [B,H,d_v] -> O
    [B,H,d_v], with the state S [B,H,d_v,d_k] updated in place; log_alpha [B,H],
    [H] or None.  Otherwise as gdn_lin_fwd."""
    if base._elsewhere(v, stream):
        with base._moved("gdn_lin_step", v, stream):
            return gdn_lin_step(q, k, v, log_alpha, S, scale, o_dtype, O)
    dev, io = v.device, v.dtype
    if S is None:
        raise ValueError("gdn_lin_step needs the state S")
    base._rank("q", q, 3)
    base._rank("k", k, 3)
    base._rank("v", v, 3)
    (B, H, dv), (_, Hq, dk), Hk = v.shape, q.shape, k.shape[1]
    if Hq < 1 or Hk < 1 or H % Hq or H % Hk:
        raise ValueError(f"{H} heads of values do not divide among {Hq} of queries and {Hk} of keys")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    # (one expression where all is well; the checks one by one say what is wrong)
    if not (q.shape == (B, Hq, dk) and k.shape == (B, Hk, dk) and S.shape == (B, H, dv, dk) and io is q.dtype is k.dtype
            and S.dtype is _F32 and dev == q.device == k.device == S.device and qs[2] == ks[2] == vs[2] == 1
            and S.is_contiguous()):
        base._check("q", q, (B, Hq, dk), io, dev, 1)
        base._check("k", k, (B, Hk, dk), io, dev, 1)
        base._check("v", v, (B, H, dv), io, dev, 1)
        base._check("S", S, (B, H, dv, dk), _F32, dev)
    per_head, a = 0, (0, 0)
    if log_alpha is not None:
        _check_decay(log_alpha, H, (B, H), dev)
        per_head, a = (1, a) if log_alpha.dim() == 1 else (0, log_alpha.stride())
    if o_dtype is None:
        o_dtype = io if O is None else O.dtype
    s = GdnLinShape(B, H, 1, Hq, Hk, dk, dv, base._code(io), base._code(o_dtype), per_head, float(scale),
                    qs[0], qs[1], 0, ks[0], ks[1], 0, vs[0], vs[1], 0, a[0], a[1], 0)
    if O is None:
        O = torch.empty((B, H, dv), dtype=o_dtype, device=dev)
    else:
        base._check("O", O, (B, H, dv), o_dtype, dev)
    check(load().gdn_lin_step(ctypes.byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), base._ptr(log_alpha), S.data_ptr(),
                              O.data_ptr(), base._stream(v)))
    return O


def gdn_lin_bwd_workspace_bytes(shape: GdnLinShape) -> int:
    return base._query("gdn_lin_bwd_workspace_bytes", shape)


def gdn_lin_bwd(dO, q, k, v, log_alpha=None, S0=None, lens=None, dS_final=None, scale=1.0, stream=None):
    """Gradient of gdn_lin_fwd: dO [B,H,T,d_v] contiguous, in v's dtype (an O
    taken in another dtype: cast its gradient), dS_final [B,H,d_v,d_k] fp32 or
    None.  Returns a dict, all contiguous: dq [B,Hq,T,d_k], dk [B,Hk,T,d_k]
    (summed over the heads that share them), dv [B,H,T,d_v] in v's dtype and, with
    the inputs they belong to, dlog_alpha fp32 ([B,H,T], or [H] summed over
    sequences and tokens; 0 where the decay is 0) and dS0 fp32."""
    if base._elsewhere(v, stream):
        with base._moved("gdn_lin_bwd", v, stream):
            return gdn_lin_bwd(dO, q, k, v, log_alpha, S0, lens, dS_final, scale)
    dev, io = v.device, v.dtype
    s = _lin_shape(q, k, v, log_alpha, scale, io)
    _lin_check(s, q, k, v, log_alpha, S0, lens, dev)
    base._check("dO", dO, (s.B, s.H, s.T, s.d_v), io, dev)
    base._check("dS_final", dS_final, (s.B, s.H, s.d_v, s.d_k), _F32, dev)
    out = {"dq": torch.empty((s.B, s.Hq, s.T, s.d_k), dtype=io, device=dev),
           "dk": torch.empty((s.B, s.Hk, s.T, s.d_k), dtype=io, device=dev),
           "dv": torch.empty((s.B, s.H, s.T, s.d_v), dtype=io, device=dev)}
    if log_alpha is not None:
        out["dlog_alpha"] = torch.empty((s.H,) if s.per_head else (s.B, s.H, s.T), dtype=_F32, device=dev)
    if S0 is not None:
        out["dS0"] = torch.empty_like(S0)
    nbytes = gdn_lin_bwd_workspace_bytes(s)
    wp, ws = base._workspace(nbytes, dev)
    check(load().gdn_lin_bwd(ctypes.byref(s), dO.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), base._ptr(log_alpha),
                             base._ptr(S0), base._ptr(dS_final), base._ptr(lens), out["dq"].data_ptr(), out["dk"].data_ptr(),
                             out["dv"].data_ptr(), base._ptr(out.get("dlog_alpha")), base._ptr(out.get("dS0")), wp, nbytes,
                             base._stream(v)))
    return out


# ---- norms around a block ----

def _block_shape(o, x, gate, act, post, eps):
    base._rank("o", o, 3)
    base._rank("x", x, 3)
    B, T, D = o.shape
    if act not in _ACTS:
        raise ValueError(f"act must be 'sigmoid', 'silu' or None, got {act!r}")
    if gate is None:
        gs = (0, 0)
    else:
        base._rank("gate", gate, 3)
        gs = gate.stride()
    os, xs = o.stride(), x.stride()
    return GdnBlockNormShape(B, T, D, base._code(o.dtype), base._code(x.dtype), 1 if post else 0, _ACTS[act], float(eps),
                             os[0], os[1], xs[0], xs[1], gs[0], gs[1])


def _block_check(s, o, x, w_pre, w_post, gate, scale, dev):
    rows = (s.B, s.T, s.D)
    base._check("o", o, rows, o.dtype, dev, 1)
    base._check("x", x, rows, x.dtype, dev, 1)
    base._check("gate", gate, rows, o.dtype, dev, 1)
    base._check("w_pre", w_pre, (s.D,), _F32, dev)
    base._check("w_post", w_post, (s.D,), _F32, dev)
    base._check("scale", scale, (s.D,), _F32, dev)
    if w_post is not None and not s.post:
        raise ValueError("w_post goes with post=True")


def gdn_block_norm_fwd(o, x, w_pre=None, w_post=None, gate=None, scale=None, act="sigmoid", post=True, pre=True, eps=1e-5,
                       x_out=None, y=None, stream=None):
    """A block's output into the residual stream, and on to the next block:
        n = o / sqrt(mean(o^2) + eps) w_post   (post=False: n = o)
        x_out = x + scale act(gate) n
        y = x_out / sqrt(mean(x_out^2) + eps) w_pre   (pre=False: no y)
    over the last dimension.  o, gate [B,T,D] of one dtype, x [B,T,D] of its own,
    bf16 or fp32, views with a contiguous last dimension (D <= 16384); w_pre,
    w_post, scale [D] fp32 or None (1); gate None: act(gate) = 1; act of the gate
    'sigmoid', 'silu' or None.  Returns (x_out [B,T,D] in x's dtype, y [B,T,D] in
    o's), which may be passed in; x_out may be x where that is contiguous."""
    if base._elsewhere(o, stream):
        with base._moved("gdn_block_norm_fwd", o, stream):
            return gdn_block_norm_fwd(o, x, w_pre, w_post, gate, scale, act, post, pre, eps, x_out, y)
    dev = o.device
    s = _block_shape(o, x, gate, act, post, eps)
    _block_check(s, o, x, w_pre, w_post, gate, scale, dev)
    rows = (s.B, s.T, s.D)
    if not pre and (w_pre is not None or y is not None):
        raise ValueError("w_pre and y go with pre=True")
    if x_out is None:
        x_out = torch.empty(rows, dtype=x.dtype, device=dev)
    else:
        base._check("x_out", x_out, rows, x.dtype, dev)
        same = x_out.data_ptr() == x.data_ptr() and x.is_contiguous()
        base._separate("x_out", x_out, o=o, x=None if same else x, gate=gate, w_pre=w_pre, w_post=w_post, scale=scale)
    if pre:
        if y is None:
            y = torch.empty(rows, dtype=o.dtype, device=dev)
        else:
            base._check("y", y, rows, o.dtype, dev)
            base._separate("y", y, o=o, x=x, gate=gate, w_pre=w_pre, w_post=w_post, scale=scale, x_out=x_out)
    check(load().gdn_block_norm_fwd(ctypes.byref(s), o.data_ptr(), x.data_ptr(), base._ptr(gate), base._ptr(w_post),
                                    base._ptr(scale), base._ptr(w_pre), x_out.data_ptr(), base._ptr(y), base._stream(o)))
    return x_out, y


def gdn_block_norm_bwd_workspace_bytes(shape: GdnBlockNormShape) -> int:
    return base._query("gdn_block_norm_bwd_workspace_bytes", shape)


def gdn_block_norm_bwd(dx_out, dy, x_out, o, w_pre=None, w_post=None, gate=None, scale=None, act="sigmoid", post=True, eps=1e-5,
                       stream=None):
    """Gradient of gdn_block_norm_fwd from the x_out that it wrote and its other
    inputs: dx_out [B,T,D] in x_out's dtype and dy [B,T,D] in o's, contiguous,
    either may be None (zero; dy where y was not taken).  Returns a dict, all
    contiguous: dx in x_out's dtype, do in o's and, with the inputs they belong
    to, dgate in o's dtype, dw_pre, dw_post, dscale [D] fp32."""
    if base._elsewhere(o, stream):
        with base._moved("gdn_block_norm_bwd", o, stream):
            return gdn_block_norm_bwd(dx_out, dy, x_out, o, w_pre, w_post, gate, scale, act, post, eps)
    dev = o.device
    s = _block_shape(o, x_out, gate, act, post, eps)
    _block_check(s, o, x_out, w_pre, w_post, gate, scale, dev)
    rows = (s.B, s.T, s.D)
    if dx_out is None and dy is None:
        raise ValueError("gdn_block_norm_bwd needs dx_out or dy")
    if dy is None and w_pre is not None:
        raise ValueError("w_pre goes with dy")
    base._check("dx_out", dx_out, rows, x_out.dtype, dev)
    base._check("dy", dy, rows, o.dtype, dev)
    out = {"dx": torch.empty(rows, dtype=x_out.dtype, device=dev), "do": torch.empty(rows, dtype=o.dtype, device=dev)}
    if gate is not None:
        out["dgate"] = torch.empty(rows, dtype=o.dtype, device=dev)
    for name, w in (("dw_pre", w_pre), ("dw_post", w_post), ("dscale", scale)):
        if w is not None:
            out[name] = torch.empty_like(w)
    nbytes = gdn_block_norm_bwd_workspace_bytes(s)
    wp, ws = base._workspace(nbytes, dev)
    check(load().gdn_block_norm_bwd(ctypes.byref(s), base._ptr(dx_out), base._ptr(dy), x_out.data_ptr(), o.data_ptr(),
                                    base._ptr(gate), base._ptr(w_post), base._ptr(scale), base._ptr(w_pre), out["dx"].data_ptr(),
                                    out["do"].data_ptr(), base._ptr(out.get("dgate")), base._ptr(out.get("dw_post")),
                                    base._ptr(out.get("dscale")), base._ptr(out.get("dw_pre")), wp, nbytes, base._stream(o)))
    return out
