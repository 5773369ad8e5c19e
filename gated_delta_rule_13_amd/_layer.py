"""Binding of the operators around the recurrence (``include/gdn.h``): the
short causal convolution, the selective state space recurrence and the head
normalisation.  Argument checks and marshalling only; every step of the
computation runs in the HIP kernels of ``libgdn.so``.

Strided inputs may be views (slices of a projection's output, transposed
heads): only their last dimension has to be contiguous, or where it is stated
the last two.  Outputs carry no autograd history, whatever their inputs
require: a model joins a call and its ``_bwd`` in an autograd function of its
own.  Calls run on ``stream`` (the current stream of the tensors'
device by default), asynchronously.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import GDN_BF16, GDN_F32, GdnConvShape, GdnError, GdnNormShape, GdnSsmShape, check, load

__all__ = ["gdn_conv_fwd", "gdn_conv_bwd", "gdn_conv_step", "gdn_conv_bwd_workspace_bytes",
           "gdn_ssm_fwd", "gdn_ssm_bwd", "gdn_ssm_step", "gdn_ssm_fwd_workspace_bytes",
           "gdn_ssm_bwd_workspace_bytes",
           "gdn_norm_fwd", "gdn_norm_bwd", "gdn_norm_bwd_workspace_bytes"]

_INT32 = 2 ** 31 - 1
_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _code(dt) -> int:
    code = _CODES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")
    return code


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _elsewhere(t, stream) -> bool:
    """Whether a call has to move to another device or stream first."""
    return stream is not None or not t.is_cuda or t.get_device() != torch.cuda.current_device()


@contextlib.contextmanager
def _moved(name, t, stream):
    """The tensors' device and the call's stream made current, so that what
    the call allocates belongs to that stream."""
    if not t.is_cuda:
        raise ValueError(f"{name} runs on the GPU: tensors must be on a cuda device")
    if stream is None:
        with torch.cuda.device(t.device):
            yield
    elif stream.device != t.device:
        raise ValueError(f"the stream must be on {t.device}, got {stream.device}")
    else:
        with torch.cuda.stream(stream):
            yield


def _stream(t) -> int:
    """Handle of the current stream (the raw handle takes 0.1 us, a Stream
    object 1.9 us: a single token's kernel runs for 3)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _check(name, t, shape, dtype, device, tail=None):
    """Shape, dtype and device of t, and that it is contiguous (tail None) or
    that its last dimension (tail 1) or two dimensions (tail 2) are."""
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if tail is None:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if tail == 2 and t.stride(-2) != shape[-1] and shape[-2] > 1:
        raise ValueError(f"the last 2 dimensions of {name} must be contiguous")


def _rank(name, t, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {t.dim()}")
    if t.numel() > _INT32 and max(t.shape) > _INT32:      # (the shape structures would wrap)
        raise ValueError(f"the dimensions of {name} must be below 2^31, got {tuple(t.shape)}")


def _separate(name, out, **inputs):
    """An output of the caller's shares no memory with an input (as far as the
    ranges of their elements tell)."""
    base = out.untyped_storage().data_ptr()
    for other, t in inputs.items():
        if t is not None and t.untyped_storage().data_ptr() == base:
            (a0, a1), (b0, b1) = _range(out), _range(t)
            if a0 < b1 and b0 < a1:
                raise ValueError(f"{name} may not overlap {other}")


def _range(t):
    span = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1
    return t.data_ptr(), t.data_ptr() + span * t.element_size()


def _query(entry, shape) -> int:
    n = getattr(load(), entry)(ctypes.byref(shape))
    if n == ctypes.c_size_t(-1).value:
        raise GdnError(4, load().gdn_last_error().decode())
    return n


def _workspace(nbytes, device):
    """(256-byte aligned pointer, tensor that owns it) of nbytes."""
    if not nbytes:
        return None, None
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    return (ws.data_ptr() + 255) // 256 * 256, ws


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
    if _elsewhere(x, stream):
        with _moved("gdn_conv_fwd", x, stream):
            return gdn_conv_fwd(x, weight, bias, state0, lens, heads, act, y, state_out)
    dev = x.device
    s = _conv_shape(x, weight, heads, act)
    _conv_check(s, x, weight, bias, state0, lens, dev)
    if y is None:
        y = x.new_empty(_conv_out_shape(s, heads))
    else:
        _check("y", y, _conv_out_shape(s, heads), x.dtype, dev)
        _separate("y", y, x=x, weight=weight, bias=bias, state0=state0, lens=lens)
    if state_out is None:
        state_out = x.new_empty((s.B, s.W - 1, s.D))
    else:
        _check("state_out", state_out, (s.B, s.W - 1, s.D), x.dtype, dev)
        same = state0 is not None and state_out.data_ptr() == state0.data_ptr()
        _separate("state_out", state_out, x=x, weight=weight, bias=bias, state0=None if same else state0, lens=lens, y=y)
    check(load().gdn_conv_fwd(ctypes.byref(s), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state0), _ptr(lens),
                              y.data_ptr(), state_out.data_ptr(), _stream(x)))
    return y, state_out


def gdn_conv_step(x, weight, bias, state, act="silu", y=None, stream=None):
    """One token of every sequence: x [B,D] -> y [B,D], with state [B,W-1,D]
    updated in place.  Otherwise as gdn_conv_fwd."""
    if _elsewhere(x, stream):
        with _moved("gdn_conv_step", x, stream):
            return gdn_conv_step(x, weight, bias, state, act, y)
    dev, io = x.device, x.dtype
    if state is None:
        raise ValueError("gdn_conv_step needs the state")
    _rank("x", x, 2)
    _rank("weight", weight, 2)
    (B, D), W = x.shape, weight.shape[1]
    _check("x", x, (B, D), io, dev, 1)
    _check("weight", weight, (D, W), torch.float32, dev)
    _check("bias", bias, (D,), torch.float32, dev)
    _check("state", state, (B, W - 1, D), io, dev)
    _separate("state", state, x=x)
    s = GdnConvShape(B, 1, D, W, 1, _code(io), _silu(act), x.stride(0), 0)
    if y is None:
        y = x.new_empty((B, D))
    else:
        _check("y", y, (B, D), io, dev)
        _separate("y", y, x=x, weight=weight, bias=bias, state=state)
    check(load().gdn_conv_step(ctypes.byref(s), x.data_ptr(), weight.data_ptr(), _ptr(bias), state.data_ptr(),
                               y.data_ptr(), _stream(x)))
    return y


def gdn_conv_bwd_workspace_bytes(shape: GdnConvShape) -> int:
    return _query("gdn_conv_bwd_workspace_bytes", shape)


def gdn_conv_bwd(dy, x, weight, bias=None, state0=None, lens=None, dstate_out=None, act="silu", stream=None):
    """Gradient of gdn_conv_fwd: dy as y ([B,T,D] or [B,heads,T,D/heads],
    contiguous), dstate_out [B,W-1,D] or None.  Returns a dict: dx [B,T,D] in
    x's dtype, dweight [D,W] and dbias [D] fp32 (dbias with a bias only),
    dstate0 [B,W-1,D] (with a state0 only)."""
    if _elsewhere(x, stream):
        with _moved("gdn_conv_bwd", x, stream):
            return gdn_conv_bwd(dy, x, weight, bias, state0, lens, dstate_out, act)
    dev = x.device
    if dy.dim() not in (3, 4):
        raise ValueError(f"dy must have 3 or 4 dimensions, got {dy.dim()}")
    heads = dy.shape[1] if dy.dim() == 4 else None
    s = _conv_shape(x, weight, heads, act)
    _conv_check(s, x, weight, bias, state0, lens, dev)
    _check("dy", dy, _conv_out_shape(s, heads), x.dtype, dev)
    _check("dstate_out", dstate_out, (s.B, s.W - 1, s.D), x.dtype, dev)
    out = {"dx": x.new_empty((s.B, s.T, s.D)), "dweight": torch.empty_like(weight)}
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    if state0 is not None:
        out["dstate0"] = torch.empty_like(state0)
    nbytes = gdn_conv_bwd_workspace_bytes(s)
    wp, ws = _workspace(nbytes, dev)
    check(load().gdn_conv_bwd(ctypes.byref(s), dy.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state0),
                              _ptr(dstate_out), _ptr(lens), out["dx"].data_ptr(), out["dweight"].data_ptr(),
                              _ptr(out.get("dbias")), _ptr(out.get("dstate0")), wp, nbytes, _stream(x)))
    return out


# ---- selective state space recurrence ----

def _ssm_shape(x, dt, A, Bm, C, z, dt_softplus):
    _rank("x", x, 3)
    _rank("dt", dt, 3)
    _rank("Bm", Bm, 4)
    _rank("C", C, 4)
    B, T, D = x.shape
    _, _, G, N = Bm.shape
    if G < 1 or D % G:
        raise ValueError(f"{D} channels do not divide into {G} groups")
    if z is None:
        zs = (0, 0)
    else:
        _rank("z", z, 3)
        zs = z.stride()
    xs, ds, bs, cs = x.stride(), dt.stride(), Bm.stride(), C.stride()
    return GdnSsmShape(B, T, D, N, G, _code(x.dtype), 1 if dt_softplus else 0, xs[0], xs[1], ds[0], ds[1],
                       zs[0], zs[1], bs[0], bs[1], cs[0], cs[1])


def _ssm_check(s, x, dt, A, Bm, C, D, z, dt_bias, h, lens, dev):
    f32, io = torch.float32, x.dtype
    B, T, Dc, N, G = s.B, s.T, s.D, s.N, s.G
    rows, bc, each = (B, T, Dc), (B, T, G, N), (Dc,)
    _check("x", x, rows, io, dev, 1)
    _check("dt", dt, rows, io, dev, 1)
    _check("z", z, rows, io, dev, 1)
    _check("A", A, (Dc, N), f32, dev)
    _check("Bm", Bm, bc, io, dev, 2)
    _check("C", C, bc, io, dev, 2)
    _check("D", D, each, f32, dev)
    _check("dt_bias", dt_bias, each, f32, dev)
    _check("h0", h, (B, Dc, N), f32, dev)
    _check("lens", lens, (B,), torch.int32, dev)


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
    if _elsewhere(x, stream):
        with _moved("gdn_ssm_fwd", x, stream):
            return gdn_ssm_fwd(x, dt, A, Bm, C, D, z, dt_bias, h0, lens, dt_softplus, y, h_final)
    dev = x.device
    s = _ssm_shape(x, dt, A, Bm, C, z, dt_softplus)
    _ssm_check(s, x, dt, A, Bm, C, D, z, dt_bias, h0, lens, dev)
    if y is None:
        y = x.new_empty((s.B, s.T, s.D))
    else:
        _check("y", y, (s.B, s.T, s.D), x.dtype, dev)
        _separate("y", y, x=x, dt=dt, A=A, Bm=Bm, C=C, D=D, z=z, dt_bias=dt_bias, h0=h0, lens=lens)
    if h_final is None:
        h_final = A.new_empty((s.B, s.D, s.N))
    else:
        _check("h_final", h_final, (s.B, s.D, s.N), torch.float32, dev)
        same = h0 is not None and h_final.data_ptr() == h0.data_ptr()
        _separate("h_final", h_final, x=x, dt=dt, A=A, Bm=Bm, C=C, D=D, z=z, dt_bias=dt_bias, h0=None if same else h0,
                  lens=lens, y=y)
    nbytes = gdn_ssm_fwd_workspace_bytes(s)
    wp, ws = _workspace(nbytes, dev)
    check(load().gdn_ssm_fwd(ctypes.byref(s), x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), C.data_ptr(),
                             _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(lens), y.data_ptr(), h_final.data_ptr(),
                             wp, nbytes, _stream(x)))
    return y, h_final


def gdn_ssm_step(x, dt, A, Bm, C, D=None, z=None, dt_bias=None, h=None, dt_softplus=True, y=None, stream=None):
    """One token of every sequence: x, dt, z [B,D], Bm, C [B,G,N] -> y [B,D],
    with the state h [B,D,N] updated in place.  Otherwise as gdn_ssm_fwd."""
    if _elsewhere(x, stream):
        with _moved("gdn_ssm_step", x, stream):
            return gdn_ssm_step(x, dt, A, Bm, C, D, z, dt_bias, h, dt_softplus, y)
    dev = x.device
    if h is None:
        raise ValueError("gdn_ssm_step needs the state h")
    _rank("x", x, 2)
    _rank("Bm", Bm, 3)
    (B, Dc), (_, G, N), io = x.shape, Bm.shape, x.dtype
    if G < 1 or Dc % G:
        raise ValueError(f"{Dc} channels do not divide into {G} groups")
    row, bc, f32 = (B, Dc), (B, G, N), torch.float32
    # (one expression where all is well, 3 us less than the checks one by one,
    # which say what is wrong)
    xs, ds, bs, cs = x.stride(), dt.stride(), Bm.stride(), C.stride()
    if not (dt.shape == row and Bm.shape == bc and C.shape == bc and A.shape == (Dc, N) and h.shape == (B, Dc, N)
            and io is dt.dtype is Bm.dtype is C.dtype and A.dtype is h.dtype is f32
            and dev == dt.device == Bm.device == C.device == A.device == h.device
            and xs[1] == ds[1] == bs[2] == cs[2] == 1 and bs[1] == cs[1] == N and A.is_contiguous() and h.is_contiguous()):
        _check("x", x, row, io, dev, 1)
        _check("dt", dt, row, io, dev, 1)
        _check("Bm", Bm, bc, io, dev, 2)
        _check("C", C, bc, io, dev, 2)
        _check("A", A, (Dc, N), f32, dev)
        _check("h", h, (B, Dc, N), f32, dev)
    _check("z", z, row, io, dev, 1)
    _check("D", D, (Dc,), f32, dev)
    _check("dt_bias", dt_bias, (Dc,), f32, dev)
    s = GdnSsmShape(B, 1, Dc, N, G, _code(io), 1 if dt_softplus else 0, xs[0], 0, ds[0], 0,
                    0 if z is None else z.stride(0), 0, bs[0], 0, cs[0], 0)
    if y is None:
        y = x.new_empty((B, Dc))
    else:
        _check("y", y, (B, Dc), io, dev)
        _separate("y", y, x=x, dt=dt, A=A, Bm=Bm, C=C, D=D, z=z, dt_bias=dt_bias, h=h)
    check(load().gdn_ssm_step(ctypes.byref(s), x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), C.data_ptr(),
                              _ptr(D), _ptr(z), _ptr(dt_bias), h.data_ptr(), y.data_ptr(), _stream(x)))
    return y


def gdn_ssm_bwd_workspace_bytes(shape: GdnSsmShape) -> int:
    return _query("gdn_ssm_bwd_workspace_bytes", shape)


def gdn_ssm_bwd(dy, x, dt, A, Bm, C, D=None, z=None, dt_bias=None, h0=None, lens=None, dh_final=None,
                dt_softplus=True, stream=None):
    """Gradient of gdn_ssm_fwd: dy [B,T,D] contiguous, dh_final [B,D,N] fp32
    or None.  Returns a dict: dx, ddt [B,T,D], dB, dC [B,T,G,N] in x's dtype, dA
    [D,N] fp32 and, with the inputs they belong to, dD, ddt_bias [D] fp32, dz
    [B,T,D], dh0 [B,D,N] fp32.  The call takes a workspace of about 0.8 N bytes
    for each token and channel (gdn_ssm_bwd_workspace_bytes), 6 times x in bf16
    at 16 states, and gives it back when it is done."""
    if _elsewhere(x, stream):
        with _moved("gdn_ssm_bwd", x, stream):
            return gdn_ssm_bwd(dy, x, dt, A, Bm, C, D, z, dt_bias, h0, lens, dh_final, dt_softplus)
    dev = x.device
    s = _ssm_shape(x, dt, A, Bm, C, z, dt_softplus)
    _ssm_check(s, x, dt, A, Bm, C, D, z, dt_bias, h0, lens, dev)
    rows, bc = (s.B, s.T, s.D), (s.B, s.T, s.G, s.N)
    _check("dy", dy, rows, x.dtype, dev)
    _check("dh_final", dh_final, (s.B, s.D, s.N), torch.float32, dev)
    out = {"dx": x.new_empty(rows), "ddt": x.new_empty(rows), "dA": torch.empty_like(A), "dB": x.new_empty(bc),
           "dC": x.new_empty(bc)}
    if D is not None:
        out["dD"] = torch.empty_like(D)
    if z is not None:
        out["dz"] = x.new_empty(rows)
    if dt_bias is not None:
        out["ddt_bias"] = torch.empty_like(dt_bias)
    if h0 is not None:
        out["dh0"] = torch.empty_like(h0)
    nbytes = gdn_ssm_bwd_workspace_bytes(s)
    wp, ws = _workspace(nbytes, dev)
    check(load().gdn_ssm_bwd(ctypes.byref(s), dy.data_ptr(), x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(),
                             C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(dh_final), _ptr(lens),
                             out["dx"].data_ptr(), out["ddt"].data_ptr(), out["dA"].data_ptr(), out["dB"].data_ptr(),
                             out["dC"].data_ptr(), _ptr(out.get("dD")), _ptr(out.get("dz")),
                             _ptr(out.get("ddt_bias")), _ptr(out.get("dh0")), wp, nbytes, _stream(x)))
    return out


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
    if _elsewhere(x, stream):
        with _moved("gdn_norm_fwd", x, stream):
            return gdn_norm_fwd(x, weight, bias, z, act, center, eps, o_dtype, y)
    dev = x.device
    if o_dtype is None:
        o_dtype = x.dtype if z is None else z.dtype
    s = _norm_shape(x, weight, bias, z, act, center, eps, o_dtype)
    _norm_check(s, x, weight, bias, z, o_dtype, dev)
    if y is None:
        y = torch.empty(x.shape, dtype=o_dtype, device=dev)
    else:
        _check("y", y, x.shape, o_dtype, dev)
        _separate("y", y, x=x, weight=weight, bias=bias, z=z)
    check(load().gdn_norm_fwd(ctypes.byref(s), x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(z), y.data_ptr(),
                              _stream(x)))
    return y


def gdn_norm_bwd_workspace_bytes(shape: GdnNormShape) -> int:
    return _query("gdn_norm_bwd_workspace_bytes", shape)


def gdn_norm_bwd(dy, x, weight=None, bias=None, z=None, act="silu", center=False, eps=1e-5, stream=None):
    """Gradient of gdn_norm_fwd: dy [B,T,G,d] contiguous, in z's dtype.
    Returns a dict: dx in x's dtype, and in x's order of dimensions in memory
    where x is dense, and, with the inputs they belong to, dweight and dbias
    fp32 (summed over the heads for weights [d]) and dz [B,T,G,d]."""
    if _elsewhere(x, stream):
        with _moved("gdn_norm_bwd", x, stream):
            return gdn_norm_bwd(dy, x, weight, bias, z, act, center, eps)
    dev, o_dtype = x.device, dy.dtype
    s = _norm_shape(x, weight, bias, z, act, center, eps, o_dtype)
    _norm_check(s, x, weight, bias, z, o_dtype, dev)
    _check("dy", dy, x.shape, o_dtype, dev)
    dx = torch.empty_like(x)            # (dense x: the same strides; else torch's choice)
    ds = dx.stride()
    if (ds[3] != 1 and s.d > 1) or any(n > 1 and v < s.d for n, v in zip(dx.shape[:3], ds)):
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        ds = dx.stride()
    out = {"dx": dx}
    if weight is not None:
        out["dweight"] = torch.empty_like(weight)
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    if z is not None:
        out["dz"] = torch.empty(x.shape, dtype=o_dtype, device=dev)
    nbytes = gdn_norm_bwd_workspace_bytes(s)
    wp, ws = _workspace(nbytes, dev)
    check(load().gdn_norm_bwd(ctypes.byref(s), dy.data_ptr(), x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(z),
                              dx.data_ptr(), ds[0], ds[1], ds[2], _ptr(out.get("dweight")), _ptr(out.get("dbias")),
                              _ptr(out.get("dz")), wp, nbytes, _stream(x)))
    return out
