"""Binding of the operators around the recurrence (``include/gdn.h``): the
short causal convolution, the selective state space recurrence and the head
normalisation.  Argument checks and marshalling only; every step of the
computation runs in the HIP kernels of ``libgdn.so``.

Strided inputs may be views (slices of a projection's output, transposed
heads): only their last dimension has to be contiguous, or where it is stated
the last two.  Calls run on ``stream`` (the current stream of the tensors'
device by default), asynchronously.
"""
from __future__ import annotations

import ctypes

from ._lib import GDN_BF16, GDN_F32, GdnConvShape, GdnError, GdnNormShape, GdnSsmShape, check, load

__all__ = ["gdn_conv_fwd", "gdn_conv_bwd", "gdn_conv_step", "gdn_conv_bwd_workspace_bytes",
           "gdn_ssm_fwd", "gdn_ssm_bwd", "gdn_ssm_step", "gdn_ssm_fwd_workspace_bytes",
           "gdn_ssm_bwd_workspace_bytes",
           "gdn_norm_fwd", "gdn_norm_bwd", "gdn_norm_bwd_workspace_bytes"]


def _torch():
    import torch
    return torch


def _code(dt) -> int:
    torch = _torch()
    if dt == torch.bfloat16:
        return GDN_BF16
    if dt == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _device(name, t):
    if t.device.type != "cuda":
        raise ValueError(f"{name} runs on the GPU: tensors must be on a cuda device")
    return t.device


def _check(name, t, shape, dtype, device, tail=None):
    """Shape, dtype and device of t, and that it is contiguous (tail None) or
    that its last `tail` dimensions are."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if tail is None:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return
    want = 1
    for dim in range(t.dim() - 1, t.dim() - 1 - tail, -1):
        if t.shape[dim] > 1 and t.stride(dim) != want:
            raise ValueError(f"the last {'dimension' if tail == 1 else f'{tail} dimensions'} of {name} "
                             "must be contiguous")
        want *= t.shape[dim]


def _rank(name, t, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")


def _separate(name, out, **inputs):
    """An output of the caller's shares no memory with an input (as far as the
    ranges of their elements tell)."""
    if out is None:
        return
    a0, a1 = _range(out)
    for other, t in inputs.items():
        if t is not None and t.device == out.device and t.numel() and out.numel():
            b0, b1 = _range(t)
            if a0 < b1 and b0 < a1:
                raise ValueError(f"{name} may not overlap {other}")


def _range(t):
    span = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1
    return t.data_ptr(), t.data_ptr() + span * t.element_size()


class _On:
    """The device of the tensors made current, and the stream's handle."""

    def __init__(self, device, stream):
        torch = _torch()
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream must be on {device}, got {stream.device}")
        self.guard = torch.cuda.device(device)
        self.stream = torch.cuda.current_stream(device) if stream is None else stream

    def __enter__(self):
        self.guard.__enter__()
        return ctypes.c_void_p(self.stream.cuda_stream)

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)


def _query(entry, shape) -> int:
    n = getattr(load(), entry)(ctypes.byref(shape))
    if n == ctypes.c_size_t(-1).value:
        raise GdnError(4, load().gdn_last_error().decode())
    return int(n)


def _workspace(nbytes, device, stream):
    """(pointer, tensor): nbytes of device memory, 256-byte aligned, that the
    call's stream owns."""
    if not nbytes:
        return None, None
    torch = _torch()
    with torch.cuda.stream(stream):
        ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    return (ws.data_ptr() + 255) // 256 * 256, ws


def _outs(stream, device, **specs):
    """Outputs made on the call's stream: name -> (shape, dtype) or None."""
    torch = _torch()
    with torch.cuda.stream(stream):
        return {k: None if v is None else torch.empty(v[0], dtype=v[1], device=device) for k, v in specs.items()}


def _silu(act) -> int:
    if act not in ("silu", None):
        raise ValueError(f"act must be 'silu' or None, got {act!r}")
    return 1 if act == "silu" else 0


# ---- short causal convolution ----

def _conv_shape(x, weight, heads, act):
    _rank("x", x, 3)
    _rank("weight", weight, 2)
    B, T, D = x.shape
    H = 1 if heads is None else int(heads)
    if H < 1 or D % H:
        raise ValueError(f"{D} channels do not divide into {H} heads")
    return GdnConvShape(B, T, D, weight.shape[1], H, _code(x.dtype), _silu(act), x.stride(0), x.stride(1))


def _conv_check(s, x, weight, bias, state, lens, dev):
    torch = _torch()
    _check("x", x, x.shape, x.dtype, dev, tail=1)
    _check("weight", weight, (s.D, s.W), torch.float32, dev)
    _check("bias", bias, (s.D,), torch.float32, dev)
    _check("state0", state, (s.B, s.W - 1, s.D), x.dtype, dev)
    _check("lens", lens, (s.B,), torch.int32, dev)


def _conv_out_shape(s, heads):
    return (s.B, s.T, s.D) if heads is None else (s.B, s.H, s.T, s.D // s.H)


def gdn_conv_fwd(x, weight, bias=None, state0=None, lens=None, heads=None, act="silu", y=None,
                 state_out=None, stream=None):
    """Causal convolution of each channel over W = 2, 3 or 4 tokens, with SiLU
    (act=None: without).  x [B,T,D] bf16 or fp32 (a view with a contiguous last
    dimension); weight [D,W], bias [D] or None fp32, the last tap on the
    current token; state0 [B,W-1,D] (the rows before x, oldest first; None:
    zero); lens [B] int32 or None, the tokens of each sequence in a padded
    batch (rows behind are written as zero).  Returns (y, state_out): y
    [B,T,D], or [B,heads,T,D/heads] as gdn_chunk_fwd takes q, k and v;
    state_out [B,W-1,D], the last W-1 rows, which may be passed in and may be
    state0 (in place)."""
    dev = _device("gdn_conv_fwd", x)
    torch = _torch()
    s = _conv_shape(x, weight, heads, act)
    _conv_check(s, x, weight, bias, state0, lens, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        made = _outs(st, dev, y=(_conv_out_shape(s, heads), x.dtype) if y is None else None,
                     state_out=((s.B, s.W - 1, s.D), x.dtype) if state_out is None else None)
        y = made["y"] if y is None else y
        _check("y", y, _conv_out_shape(s, heads), x.dtype, dev)
        if state_out is None:
            state_out = made["state_out"]
        else:
            _check("state_out", state_out, (s.B, s.W - 1, s.D), x.dtype, dev)
            same = state0 is not None and state_out.data_ptr() == state0.data_ptr()
            _separate("state_out", state_out, x=x, y=y, state0=None if same else state0)
        _separate("y", y, x=x, state0=state0)
        check(load().gdn_conv_fwd(ctypes.byref(s), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state0), _ptr(lens),
                                  _ptr(y), _ptr(state_out), hs))
    return y, state_out


def gdn_conv_step(x, weight, bias, state, act="silu", y=None, stream=None):
    """One token of every sequence: x [B,D] -> y [B,D], with state [B,W-1,D]
    updated in place.  Otherwise as gdn_conv_fwd."""
    dev = _device("gdn_conv_step", x)
    _rank("x", x, 2)
    torch = _torch()
    row = x.unsqueeze(1)
    s = _conv_shape(row, weight, None, act)
    if state is None:
        raise ValueError("gdn_conv_step needs the state")
    _conv_check(s, row, weight, bias, state, None, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        if y is None:
            y = _outs(st, dev, y=((s.B, s.D), x.dtype))["y"]
        else:
            _check("y", y, (s.B, s.D), x.dtype, dev)
            _separate("y", y, x=x, state=state)
        _separate("state", state, x=x)
        check(load().gdn_conv_step(ctypes.byref(s), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(y), hs))
    return y


def gdn_conv_bwd_workspace_bytes(shape: GdnConvShape) -> int:
    return _query("gdn_conv_bwd_workspace_bytes", shape)


def gdn_conv_bwd(dy, x, weight, bias=None, state0=None, lens=None, dstate_out=None, act="silu", stream=None):
    """Gradient of gdn_conv_fwd: dy as y ([B,T,D] or [B,heads,T,D/heads],
    contiguous), dstate_out [B,W-1,D] or None.  Returns a dict: dx [B,T,D] in
    x's dtype, dweight [D,W] and dbias [D] fp32 (dbias with a bias only),
    dstate0 [B,W-1,D] (with a state0 only)."""
    dev = _device("gdn_conv_bwd", x)
    torch = _torch()
    if dy.dim() not in (3, 4):
        raise ValueError(f"dy must have 3 or 4 dimensions, got {dy.dim()}")
    heads = dy.shape[1] if dy.dim() == 4 else None
    s = _conv_shape(x, weight, heads, act)
    _conv_check(s, x, weight, bias, state0, lens, dev)
    _check("dy", dy, _conv_out_shape(s, heads), x.dtype, dev)
    _check("dstate_out", dstate_out, (s.B, s.W - 1, s.D), x.dtype, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        out = _outs(st, dev, dx=((s.B, s.T, s.D), x.dtype), dweight=((s.D, s.W), torch.float32),
                    dbias=None if bias is None else ((s.D,), torch.float32),
                    dstate0=None if state0 is None else ((s.B, s.W - 1, s.D), x.dtype))
        nbytes = gdn_conv_bwd_workspace_bytes(s)
        wp, ws = _workspace(nbytes, dev, st)
        check(load().gdn_conv_bwd(ctypes.byref(s), _ptr(dy), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state0),
                                  _ptr(dstate_out), _ptr(lens), _ptr(out["dx"]), _ptr(out["dweight"]),
                                  _ptr(out["dbias"]), _ptr(out["dstate0"]), wp, nbytes, hs))
    return {k: v for k, v in out.items() if v is not None}


# ---- selective state space recurrence ----

def _ssm_shape(x, dt, A, Bm, C, z, dt_softplus):
    for name, t, n in (("x", x, 3), ("dt", dt, 3), ("A", A, 2), ("Bm", Bm, 4), ("C", C, 4)):
        _rank(name, t, n)
    if z is not None:
        _rank("z", z, 3)
    B, T, D = x.shape
    G, N = Bm.shape[2:]
    if G < 1 or D % G:
        raise ValueError(f"{D} channels do not divide into {G} groups")
    strides = []
    for t in (x, dt, z, Bm, C):
        strides += [0, 0] if t is None else [t.stride(0), t.stride(1)]
    return GdnSsmShape(B, T, D, N, G, _code(x.dtype), 1 if dt_softplus else 0, *strides)


def _ssm_check(s, x, dt, A, Bm, C, D, z, dt_bias, h, lens, dev):
    torch = _torch()
    f32, io = torch.float32, x.dtype
    rows = (s.B, s.T, s.D)
    _check("x", x, rows, io, dev, tail=1)
    _check("dt", dt, rows, io, dev, tail=1)
    _check("z", z, rows, io, dev, tail=1)
    _check("A", A, (s.D, s.N), f32, dev)
    _check("Bm", Bm, (s.B, s.T, s.G, s.N), io, dev, tail=2)
    _check("C", C, (s.B, s.T, s.G, s.N), io, dev, tail=2)
    _check("D", D, (s.D,), f32, dev)
    _check("dt_bias", dt_bias, (s.D,), f32, dev)
    _check("h0", h, (s.B, s.D, s.N), f32, dev)
    _check("lens", lens, (s.B,), torch.int32, dev)


def gdn_ssm_fwd_workspace_bytes(shape: GdnSsmShape) -> int:
    return _query("gdn_ssm_fwd_workspace_bytes", shape)


def gdn_ssm_fwd(x, dt, A, Bm, C, D=None, z=None, dt_bias=None, h0=None, lens=None, dt_softplus=True, y=None,
                h_final=None, stream=None):
    """Selective state space recurrence:
        s = softplus(dt + dt_bias),  h_t = exp(s_t A) h_{t-1} + s_t x_t Bm_t,
        y_t = (C_t . h_t + D x_t) silu(z_t).
    x, dt, z [B,T,D], Bm, C [B,T,G,N] (G groups of D/G channels, N <= 64) of
    one dtype, bf16 or fp32, views with contiguous rows; A [D,N], D, dt_bias
    [D] fp32 (D, z, dt_bias may be None); h0 [B,D,N] fp32 or None (zero); lens
    [B] int32 or None (rows behind a sequence's length are written as zero);
    dt_softplus=False takes dt + dt_bias as it is.  Returns (y [B,T,D] in x's
    dtype, h_final [B,D,N] fp32), which may be passed in; h_final may be h0."""
    dev = _device("gdn_ssm_fwd", x)
    torch = _torch()
    s = _ssm_shape(x, dt, A, Bm, C, z, dt_softplus)
    _ssm_check(s, x, dt, A, Bm, C, D, z, dt_bias, h0, lens, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        made = _outs(st, dev, y=((s.B, s.T, s.D), x.dtype) if y is None else None,
                     h=((s.B, s.D, s.N), torch.float32) if h_final is None else None)
        if y is None:
            y = made["y"]
        else:
            _check("y", y, (s.B, s.T, s.D), x.dtype, dev)
            _separate("y", y, x=x, dt=dt, z=z, Bm=Bm, C=C)
        if h_final is None:
            h_final = made["h"]
        else:
            _check("h_final", h_final, (s.B, s.D, s.N), torch.float32, dev)
            same = h0 is not None and h_final.data_ptr() == h0.data_ptr()
            _separate("h_final", h_final, h0=None if same else h0, x=x, dt=dt, A=A, y=y)
        nbytes = gdn_ssm_fwd_workspace_bytes(s)
        wp, ws = _workspace(nbytes, dev, st)
        check(load().gdn_ssm_fwd(ctypes.byref(s), _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(C), _ptr(D), _ptr(z),
                                 _ptr(dt_bias), _ptr(h0), _ptr(lens), _ptr(y), _ptr(h_final), wp, nbytes, hs))
    return y, h_final


def gdn_ssm_step(x, dt, A, Bm, C, D=None, z=None, dt_bias=None, h=None, dt_softplus=True, y=None, stream=None):
    """One token of every sequence: x, dt, z [B,D], Bm, C [B,G,N] -> y [B,D],
    with the state h [B,D,N] updated in place.  Otherwise as gdn_ssm_fwd."""
    dev = _device("gdn_ssm_step", x)
    torch = _torch()
    if h is None:
        raise ValueError("gdn_ssm_step needs the state h")
    _rank("x", x, 2)
    row = [None if t is None else t.unsqueeze(1) for t in (x, dt, Bm, C, z)]
    s = _ssm_shape(row[0], row[1], A, row[2], row[3], row[4], dt_softplus)
    _ssm_check(s, row[0], row[1], A, row[2], row[3], D, row[4], dt_bias, h, None, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        if y is None:
            y = _outs(st, dev, y=((s.B, s.D), x.dtype))["y"]
        else:
            _check("y", y, (s.B, s.D), x.dtype, dev)
            _separate("y", y, x=x, dt=dt, z=z, Bm=Bm, C=C, h=h)
        check(load().gdn_ssm_step(ctypes.byref(s), _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(C), _ptr(D), _ptr(z),
                                  _ptr(dt_bias), _ptr(h), _ptr(y), hs))
    return y


def gdn_ssm_bwd_workspace_bytes(shape: GdnSsmShape) -> int:
    return _query("gdn_ssm_bwd_workspace_bytes", shape)


def gdn_ssm_bwd(dy, x, dt, A, Bm, C, D=None, z=None, dt_bias=None, h0=None, lens=None, dh_final=None,
                dt_softplus=True, stream=None):
    """Gradient of gdn_ssm_fwd: dy [B,T,D] contiguous, dh_final [B,D,N] fp32
    or None.  Returns a dict: dx, ddt [B,T,D], dB, dC [B,T,G,N] in x's dtype, dA
    [D,N] fp32 and, with the inputs they belong to, dD, ddt_bias [D] fp32, dz
    [B,T,D], dh0 [B,D,N] fp32."""
    dev = _device("gdn_ssm_bwd", x)
    torch = _torch()
    s = _ssm_shape(x, dt, A, Bm, C, z, dt_softplus)
    _ssm_check(s, x, dt, A, Bm, C, D, z, dt_bias, h0, lens, dev)
    rows, state, f32 = (s.B, s.T, s.D), (s.B, s.D, s.N), torch.float32
    _check("dy", dy, rows, x.dtype, dev)
    _check("dh_final", dh_final, state, f32, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        out = _outs(st, dev, dx=(rows, x.dtype), ddt=(rows, x.dtype), dA=((s.D, s.N), f32),
                    dB=((s.B, s.T, s.G, s.N), x.dtype), dC=((s.B, s.T, s.G, s.N), x.dtype),
                    dD=None if D is None else ((s.D,), f32), dz=None if z is None else (rows, x.dtype),
                    ddt_bias=None if dt_bias is None else ((s.D,), f32), dh0=None if h0 is None else (state, f32))
        nbytes = gdn_ssm_bwd_workspace_bytes(s)
        wp, ws = _workspace(nbytes, dev, st)
        check(load().gdn_ssm_bwd(ctypes.byref(s), _ptr(dy), _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(C), _ptr(D),
                                 _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(dh_final), _ptr(lens),
                                 _ptr(out["dx"]), _ptr(out["ddt"]), _ptr(out["dA"]), _ptr(out["dB"]),
                                 _ptr(out["dC"]), _ptr(out["dD"]), _ptr(out["dz"]), _ptr(out["ddt_bias"]),
                                 _ptr(out["dh0"]), wp, nbytes, hs))
    return {k: v for k, v in out.items() if v is not None}


# ---- head normalisation ----

def _norm_shape(x, weight, bias, z, act, center, eps, o_dtype):
    _rank("x", x, 4)
    B, T, G, d = x.shape
    per_group = [t.dim() == 2 for t in (weight, bias) if t is not None]
    if len(set(per_group)) > 1:
        raise ValueError("weight and bias must both be [d] or both [G, d]")
    zs = [0, 0, 0] if z is None else list(z.stride()[:3])
    return GdnNormShape(B, T, G, d, _code(x.dtype), _code(o_dtype), 1 if center else 0,
                        1 if any(per_group) else 0, _silu(act), float(eps), *x.stride()[:3], *zs)


def _norm_check(s, x, weight, bias, z, o_dtype, dev):
    torch = _torch()
    _check("x", x, x.shape, x.dtype, dev, tail=1)
    wshape = (s.G, s.d) if s.w_per_group else (s.d,)
    _check("weight", weight, wshape, torch.float32, dev)
    _check("bias", bias, wshape, torch.float32, dev)
    _check("z", z, x.shape, o_dtype, dev, tail=1)


def gdn_norm_fwd(x, weight=None, bias=None, z=None, act="silu", center=False, eps=1e-5, o_dtype=None, y=None,
                 stream=None):
    """Normalisation of each head of each token, with an activation or a gate:
        n = (x - mean) / sqrt(var + eps) over d  (center=False: mean 0),
        y = (n weight + bias) act(z), or act(n weight + bias) without z.
    x [B,T,G,d] bf16 or fp32, a view with a contiguous last dimension (the
    delta rule's O [B,H,T,d] as O.transpose(1, 2)); weight, bias fp32 [d] for
    all heads or [G,d], or None; z [B,T,G,d] in o_dtype, a view.  Returns y
    [B,T,G,d] contiguous in o_dtype (default: z's dtype, or x's)."""
    dev = _device("gdn_norm_fwd", x)
    torch = _torch()
    if o_dtype is None:
        o_dtype = x.dtype if z is None else z.dtype
    s = _norm_shape(x, weight, bias, z, act, center, eps, o_dtype)
    _norm_check(s, x, weight, bias, z, o_dtype, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        if y is None:
            y = _outs(st, dev, y=(tuple(x.shape), o_dtype))["y"]
        else:
            _check("y", y, x.shape, o_dtype, dev)
            _separate("y", y, x=x, z=z)
        check(load().gdn_norm_fwd(ctypes.byref(s), _ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ptr(y), hs))
    return y


def gdn_norm_bwd_workspace_bytes(shape: GdnNormShape) -> int:
    return _query("gdn_norm_bwd_workspace_bytes", shape)


def gdn_norm_bwd(dy, x, weight=None, bias=None, z=None, act="silu", center=False, eps=1e-5, stream=None):
    """Gradient of gdn_norm_fwd: dy [B,T,G,d] contiguous, in z's dtype.
    Returns a dict: dx in x's dtype, and in x's order of dimensions in memory
    where x is dense, and, with the inputs they belong to, dweight and dbias
    fp32 (summed over the heads for weights [d]) and dz [B,T,G,d]."""
    dev = _device("gdn_norm_bwd", x)
    torch = _torch()
    o_dtype = dy.dtype
    s = _norm_shape(x, weight, bias, z, act, center, eps, o_dtype)
    _norm_check(s, x, weight, bias, z, o_dtype, dev)
    _check("dy", dy, x.shape, o_dtype, dev)
    st = torch.cuda.current_stream(dev) if stream is None else stream
    with _On(dev, stream) as hs:
        with torch.cuda.stream(st):
            dx = torch.empty_like(x)        # (dense x: the same strides; else contiguous)
            if dx.stride(-1) != 1 and dx.shape[-1] > 1 or any(
                    n > 1 and v < s.d for n, v in zip(dx.shape[:3], dx.stride()[:3])):
                dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        out = _outs(st, dev, dweight=None if weight is None else (tuple(weight.shape), torch.float32),
                    dbias=None if bias is None else (tuple(bias.shape), torch.float32),
                    dz=None if z is None else (tuple(x.shape), o_dtype))
        nbytes = gdn_norm_bwd_workspace_bytes(s)
        wp, ws = _workspace(nbytes, dev, st)
        check(load().gdn_norm_bwd(ctypes.byref(s), _ptr(dy), _ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ptr(dx),
                                  *dx.stride()[:3], _ptr(out["dweight"]), _ptr(out["dbias"]), _ptr(out["dz"]), wp,
                                  nbytes, hs))
    return {"dx": dx, **{k: v for k, v in out.items() if v is not None}}
