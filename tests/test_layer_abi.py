"""The C ABI of the operators around the recurrence, on the CPU: bad arguments
are refused before any launch (every call here fails validation), workspace
queries follow the shapes, and the 64-bit reference of the GPU tests agrees
with closed forms and with differences."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_13_amd as gdn
from gated_delta_rule_13_amd import _lib
from tests import layer_ref as ref
from tests.test_abi import FAKE, HEADER, lib, lib_nogpu  # noqa: F401
from tests.test_sanitizers import ROOT, clang_asan_runtime, run_child

BIG = ctypes.c_size_t(-1).value


def conv_shape(**kw):
    base = dict(B=2, T=100, D=64, W=4, H=2, dtype=0, silu=1, x_stride_b=6400, x_stride_t=64)
    return _lib.GdnConvShape(**{**base, **kw})


def ssm_shape(**kw):
    base = dict(B=2, T=100, D=64, N=16, G=2, dtype=0, dt_softplus=1)
    for n in ("x", "dt", "z"):
        base.update({n + "_stride_b": 6400, n + "_stride_t": 64})
    for n in ("b", "c"):
        base.update({n + "_stride_b": 3200, n + "_stride_t": 32})
    return _lib.GdnSsmShape(**{**base, **kw})


def norm_shape(**kw):
    base = dict(B=2, T=100, G=3, d=64, x_dtype=1, o_dtype=0, center=0, w_per_group=0, silu=1, eps=1e-5)
    for n in ("x", "z"):
        base.update({n + "_stride_b": 19200, n + "_stride_t": 192, n + "_stride_g": 64})
    return _lib.GdnNormShape(**{**base, **kw})


CALLS = {  # entry: (shape, pointer names in order, required, optional)
    "gdn_conv_fwd": (conv_shape, "x weight bias state0 lens y state_out", "x weight y"),
    "gdn_conv_step": (lambda **k: conv_shape(**{"T": 1, **k}), "x weight bias state y", "x weight state y"),
    "gdn_conv_bwd": (conv_shape, "dy x weight bias state0 dstate_out lens dx dweight dbias dstate0", "dy x weight dx dweight"),
    "gdn_ssm_fwd": (ssm_shape, "x dt A Bm C Dskip z dt_bias h0 lens y h_final", "x dt A Bm C y"),
    "gdn_ssm_step": (lambda **k: ssm_shape(**{"T": 1, **k}), "x dt A Bm C Dskip z dt_bias h y", "x dt A Bm C h y"),
    "gdn_ssm_bwd": (ssm_shape, "dy x dt A Bm C Dskip z dt_bias h0 dh_final lens dx ddt dA dBm dC dDskip dz ddt_bias dh0",
                    "dy x dt A Bm C dx ddt dA dBm dC dz"),
    "gdn_norm_fwd": (norm_shape, "x weight bias z y", "x y"),
    "gdn_norm_bwd": (norm_shape, "dy x weight bias z dx dweight dbias dz", "dy x dx dz"),
}
WORKSPACE = {"gdn_conv_bwd", "gdn_ssm_fwd", "gdn_ssm_bwd", "gdn_norm_bwd"}


def call(lib, entry, shape, ws=None, ws_bytes=0, strides=(19200, 192, 64), **ptrs):  # noqa: F811
    """The entry with fake pointers.  Where it takes a workspace, the default
    gives none, so that even a check that wrongly passed could not launch."""
    args = [ctypes.byref(shape) if shape is not None else None]
    for name in CALLS[entry][1].split():
        args.append(ptrs.get(name, FAKE))
        if entry == "gdn_norm_bwd" and name == "dx":
            args += list(strides)
    if entry in WORKSPACE:
        args += [ws, ws_bytes]
    return getattr(lib, entry)(*args, None)


ODD = ctypes.c_void_p(0x10001)     # no dtype's alignment: refused whatever else passes

BAD_CONV = [(dict(B=0), 2), (dict(T=0), 2), (dict(D=0), 2), (dict(H=0), 2), (dict(H=3), 2), (dict(dtype=2), 3),
            (dict(W=1), 4), (dict(W=5), 4), (dict(silu=2), 4), (dict(x_stride_t=-1), 2),
            (dict(B=2 ** 31 - 1, T=2 ** 31 - 1, D=2 ** 31 - 2), 2)]
BAD_SSM = [(dict(B=0), 2), (dict(T=-1), 2), (dict(D=0), 2), (dict(N=0), 2), (dict(G=0), 2), (dict(G=3), 2),
           (dict(dtype=-1), 3), (dict(N=65), 4), (dict(dt_softplus=3), 4), (dict(z_stride_b=-1), 2),
           (dict(c_stride_t=-5), 2), (dict(B=2 ** 30, T=2 ** 20, D=2), 2), (dict(D=2 ** 25), 4),
           (dict(G=2 ** 22, D=2 ** 22, B=1000), 4)]
BAD_NORM = [(dict(B=0), 2), (dict(T=0), 2), (dict(G=0), 2), (dict(d=0), 2), (dict(x_dtype=5), 3), (dict(o_dtype=-1), 3),
            (dict(d=4097), 4), (dict(center=2), 4), (dict(w_per_group=-1), 4), (dict(silu=4), 4), (dict(eps=0.0), 2),
            (dict(eps=float("nan")), 2), (dict(x_stride_g=-1), 2), (dict(z_stride_t=-1), 2)]


@pytest.mark.parametrize("entry,kw,status", [(e, kw, st) for e in CALLS for kw, st in
                                             (BAD_CONV if "conv" in e else BAD_SSM if "ssm" in e else BAD_NORM)])
def test_bad_shapes(lib_nogpu, entry, kw, status):  # noqa: F811
    assert call(lib_nogpu, entry, CALLS[entry][0](**kw), x=ODD) == status
    assert lib_nogpu.gdn_last_error().decode() != ""
    if entry in WORKSPACE:
        assert getattr(lib_nogpu, entry + "_workspace_bytes")(ctypes.byref(CALLS[entry][0](**kw))) == BIG


@pytest.mark.parametrize("entry", list(CALLS))
def test_missing_and_misaligned_arguments(lib_nogpu, entry):  # noqa: F811
    shape, names, required = CALLS[entry]
    assert call(lib_nogpu, entry, None) == 1
    for name in required.split():
        # (another argument misaligned: nothing can launch)
        other = "x" if name != "x" else required.split()[-1]
        assert call(lib_nogpu, entry, shape(), **{name: None, other: ODD}) == 1, name
    for name in names.split():
        assert call(lib_nogpu, entry, shape(), **{name: ODD}) == 4, name
    if "step" in entry:
        assert call(lib_nogpu, entry, shape(T=2), x=ODD) == 2


def test_far_rows(lib_nogpu):  # noqa: F811
    """Strides of tokens past what a group's 32-bit offsets reach."""
    for name in ("x", "dt", "z", "b", "c"):
        kw = {name + "_stride_t": 2 ** 24 + 1}
        assert call(lib_nogpu, "gdn_ssm_fwd", ssm_shape(**kw), x=ODD) == 4
        assert "strides" in lib_nogpu.gdn_last_error().decode()
        assert lib_nogpu.gdn_ssm_fwd_workspace_bytes(ctypes.byref(ssm_shape(T=1, **kw))) == 0
    assert call(lib_nogpu, "gdn_ssm_step", ssm_shape(T=1, B=65536)) == 4


@pytest.mark.parametrize("entry,kw", [
    ("gdn_conv_bwd", dict(D=2 ** 25 + 2)), ("gdn_ssm_bwd", dict(B=1100, T=1, D=32768, N=64, G=1)),
    ("gdn_ssm_fwd", dict(B=2 ** 16, D=2 ** 11, G=2 ** 11)),
    ("gdn_ssm_bwd", dict(B=64, T=2 ** 24, D=4096)), ("gdn_ssm_bwd", dict(B=64, T=2 ** 20, D=64, N=64, G=2)),
    ("gdn_norm_bwd", dict(G=2 ** 24)), ("gdn_norm_bwd", dict(G=2 ** 20, d=256, w_per_group=1))])
def test_launch_limits(lib_nogpu, entry, kw):  # noqa: F811
    """More threads than a launch counts, refused by the query and the call."""
    assert getattr(lib_nogpu, entry + "_workspace_bytes")(ctypes.byref(CALLS[entry][0](**kw))) == BIG
    assert call(lib_nogpu, entry, CALLS[entry][0](**kw), dx=ODD, y=ODD) == 4
    assert "aligned" not in lib_nogpu.gdn_last_error().decode()


def test_large_states(lib_nogpu):  # noqa: F811
    """What one pass over the tokens takes, where chains of segments would not fit."""
    big = dict(B=1100, D=32768, N=64, G=1)
    assert lib_nogpu.gdn_ssm_fwd_workspace_bytes(ctypes.byref(ssm_shape(T=1, **big))) == 0
    assert call(lib_nogpu, "gdn_ssm_step", ssm_shape(T=1, **big), x=ODD) == 4
    assert "aligned" in lib_nogpu.gdn_last_error().decode()


def test_gradient_of_one_token_keeps_no_groups(lib_nogpu):  # noqa: F811
    """Its workspace: a state, its gradient and dA for 64 lanes, dB and dC of
    each tile of channels, and 3 numbers a lane."""
    s = ssm_shape(B=128, T=1, D=4096, N=64, G=1)
    lanes, tiles = 128 * 4096, 64
    want = lanes * (3 * 64 + 3) * 4 + tiles * 128 * 2 * 64 * 4
    assert lib_nogpu.gdn_ssm_bwd_workspace_bytes(ctypes.byref(s)) == want


def test_gradient_of_the_gate_goes_with_the_gate(lib_nogpu):  # noqa: F811
    for entry in ("gdn_ssm_bwd", "gdn_norm_bwd"):
        assert call(lib_nogpu, entry, CALLS[entry][0](), z=None, x=ODD) == 1
        assert call(lib_nogpu, entry, CALLS[entry][0](), dz=None, x=ODD) == 1


def test_overlapping_rows_of_a_gradient(lib_nogpu):  # noqa: F811
    for strides in ((0, 192, 64), (19200, 63, 64), (19200, 192, 0)):
        assert call(lib_nogpu, "gdn_norm_bwd", norm_shape(), strides=strides, x=ODD) == 2


@pytest.mark.parametrize("entry", sorted(WORKSPACE))
def test_workspaces(lib_nogpu, entry):  # noqa: F811
    shape = CALLS[entry][0](T=4000)
    need = getattr(lib_nogpu, entry + "_workspace_bytes")(ctypes.byref(shape))
    assert 0 < need < BIG and need % 256 == 0
    good = ctypes.c_void_p(0x100000)
    assert call(lib_nogpu, entry, shape) == 5
    assert call(lib_nogpu, entry, shape, good, need - 1) == 5
    assert call(lib_nogpu, entry, shape, ctypes.c_void_p(0x100010), need) == 4


def test_structs_match_the_header():
    """Field names and order of the ctypes structures are the header's."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, cls in (("gdn_conv_shape", _lib.GdnConvShape), ("gdn_ssm_shape", _lib.GdnSsmShape),
                      ("gdn_norm_shape", _lib.GdnNormShape)):
        end = text.index("} " + name + ";")
        body = text[text.rindex("typedef struct {", 0, end) + 16:end]
        want = []
        for line in body.split(";"):
            words = line.replace(",", " ").split()
            if words:
                want += [(w, {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}[words[0]])
                         for w in words[1:]]
        assert want == list(cls._fields_), name


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_conv_fwd(x, w)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_conv_bwd(x, x, w)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_conv_step(x[:, 0], w, None, torch.zeros(1, 3, 8))
    bc = torch.zeros(1, 4, 1, 4)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_ssm_fwd(x, x, w, bc, bc)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_ssm_bwd(x, x, x, w, bc, bc)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_ssm_step(x[:, 0], x[:, 0], w, bc[:, 0], bc[:, 0], h=torch.zeros(1, 8, 4))
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_norm_fwd(x[None])
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_norm_bwd(x[None], x[None])


def test_api_validation_under_asan_ubsan(tmp_path):
    """This file against a build whose host code of the entry points is
    instrumented (the device code is built as usual)."""
    if os.environ.get("GDN_TEST_LIB"):
        pytest.skip("already the instrumented run")
    from gated_delta_rule_13_amd import build as b
    rt = clang_asan_runtime()
    if rt is None or shutil.which(b.hipcc()) is None:
        pytest.skip("no clang sanitizer runtime in this ROCm")
    objs = [os.path.join(b.BUILD, u[0]) for u in b.units() if u[0] != "gdn_api_layer.o"]
    if not all(os.path.exists(o) for o in objs):
        b.build()
    api = str(tmp_path / "api.o")
    cmd = [b.hipcc(), f"--offload-arch={b.ARCH}", "-O1", "-g", "-std=c++17", "-fPIC", "-fno-omit-frame-pointer",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           f"-I{b.INCLUDE}", f"-I{b.CSRC}", "-c", os.path.join(b.CSRC, "gdn_api_layer.hip"), "-o", api]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    path = str(tmp_path / "libgdn_san.so")
    res = subprocess.run([b.hipcc(), f"--offload-arch={b.ARCH}", "-shared", "-fPIC", api, *objs, "-o", path],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    out = run_child(["-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_layer_abi.py"],
                    {"LD_PRELOAD": rt, "GDN_TEST_LIB": path, "HIP_VISIBLE_DEVICES": "", "PYTHONPATH": ROOT})
    assert " passed" in out and " failed" not in out, out[-3000:]


# ---- the 64-bit reference itself ----

def test_reference_convolution_is_torchs():
    g = ref.gen(1)
    x, w, b = (ref.rand(g, *s).double() for s in ((2, 11, 6), (6, 4), (6,)))
    y, st = ref.conv(x, w, b, act=None)
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (3, 0)), w[:, None], b, groups=6)
    assert torch.allclose(y, want.transpose(1, 2), atol=1e-12)
    assert torch.equal(st, x[:, -3:])
    again, _ = ref.conv(x[:, 5:], w, b, state0=x[:, 2:5], act=None)
    assert torch.allclose(again, y[:, 5:], atol=1e-12)


def test_reference_recurrence_in_closed_form():
    """h_t = sum over r <= t of exp(A (S_t - S_r)) s_r x_r B_r."""
    g = ref.gen(2)
    x, dt = ref.rand(g, 1, 9, 3).double(), ref.rand(g, 1, 9, 3).double()
    A, Bm, C = -ref.rand(g, 3, 2).double().abs(), ref.rand(g, 1, 9, 1, 2).double(), ref.rand(g, 1, 9, 1, 2).double()
    y, h = ref.ssm(x, dt, A, Bm, C)
    s = torch.log1p(torch.exp(dt))
    S = s.cumsum(1)
    for t in range(9):
        ht = sum(torch.exp(A * (S[0, t] - S[0, r])[:, None]) * (s[0, r] * x[0, r])[:, None] * Bm[0, r] for r in range(t + 1))
        assert torch.allclose((ht * C[0, t]).sum(-1), y[0, t], atol=1e-12)
    assert torch.allclose(ht, h[0], atol=1e-12)
    part = torch.tensor([4], dtype=torch.int32)
    # (exp over tensors of different lengths may differ in its last bit: four
    # steps of numbers near 1, a few 2^-53 each)
    short = ref.ssm(x[:, :4], dt[:, :4], A, Bm[:, :4], C[:, :4])[1]
    assert torch.allclose(ref.ssm(x, dt, A, Bm, C, lens=part)[1], short, rtol=0, atol=1e-14)


def test_reference_gradients_against_differences():
    g = ref.gen(3)
    a = {"x": ref.rand(g, 1, 6, 4).double(), "dt": ref.rand(g, 1, 6, 4).double(), "A": -ref.rand(g, 4, 3).double().abs(),
         "Bm": ref.rand(g, 1, 6, 2, 3).double(), "C": ref.rand(g, 1, 6, 2, 3).double(), "z": ref.rand(g, 1, 6, 4).double()}
    dy = ref.rand(g, 1, 6, 4).double()
    grads = ref.gradients(ref.ssm, a, list(a), (dy, None))
    for n in a:
        v = ref.rand(g, *a[n].shape).double()
        assert abs(float((grads[n] * v).sum()) - ref.difference(ref.ssm, a, n, v, (dy, None))) < 1e-6
