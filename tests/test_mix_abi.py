"""The C ABI and the binding of linear attention with decay and of the norms
around a block, on the CPU: bad arguments are refused before any launch (every
call here fails), workspace queries follow the shapes, and the 64-bit references
of the GPU tests agree with closed forms and differences."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import gated_delta_rule_13_amd as gdn
from gated_delta_rule_13_amd import _layer, _lib, _mix
from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.test_abi import FAKE, HEADER, lib, lib_nogpu  # noqa: F401
from tests.test_sanitizers import ROOT, clang_asan_runtime, run_child

BIG = ctypes.c_size_t(-1).value
ODD = ctypes.c_void_p(0x10001)     # no dtype's alignment: refused whatever else passes


def lin_shape(**kw):
    base = dict(B=2, H=4, T=100, Hq=2, Hk=4, d_k=64, d_v=32, dtype=0, o_dtype=0, per_head=0, scale=1.0)
    for n, h, d in (("q", 2, 64), ("k", 4, 64), ("v", 4, 32), ("a", 4, 1)):
        base.update({n + "_stride_b": 100 * h * d, n + "_stride_h": d, n + "_stride_t": h * d})
    return _lib.GdnLinShape(**{**base, **kw})


def block_shape(**kw):
    base = dict(B=2, T=100, D=64, dtype=0, x_dtype=1, post=1, act=1, eps=1e-5)
    for n in "oxg":
        base.update({n + "_stride_b": 6400, n + "_stride_t": 64})
    return _lib.GdnBlockNormShape(**{**base, **kw})


CALLS = {  # entry: (shape, pointer names in order, required)
    "gdn_lin_fwd": (lin_shape, "q k v log_alpha S0 lens O S_final", "q k v O"),
    "gdn_lin_step": (lambda **k: lin_shape(**{"T": 1, **k}), "q k v log_alpha S O", "q k v S O"),
    "gdn_lin_bwd": (lin_shape, "dO q k v log_alpha S0 dS_final lens dq dk dv dlog_alpha dS0", "dO q k v dq dk dv"),
    "gdn_block_norm_fwd": (block_shape, "o x gate w_post scale w_pre x_out y", "o x x_out"),
    "gdn_block_norm_bwd": (block_shape, "dx_out dy x_out o gate w_post scale w_pre dx dO dgate dw_post dscale dw_pre",
                           "x_out o dx dO dgate"),
}
WORKSPACE = {"gdn_lin_fwd", "gdn_lin_bwd", "gdn_block_norm_bwd"}


def call(lib, entry, shape, ws=None, ws_bytes=0, **ptrs):  # noqa: F811
    """The entry with fake pointers, and no workspace unless one is given.  (A
    check that wrongly passed could launch only without a workspace: those calls
    here have a misaligned pointer.)"""
    args = [ctypes.byref(shape) if shape is not None else None]
    args += [ptrs.get(name, FAKE) for name in CALLS[entry][1].split()]
    if entry in WORKSPACE:
        args += [ws, ws_bytes]
    return getattr(lib, entry)(*args, None)


BAD_LIN = [(dict(B=0), 2), (dict(H=0), 2), (dict(T=0), 2), (dict(Hq=0), 2), (dict(Hk=-1), 2), (dict(Hq=3), 2), (dict(Hk=8), 2),
           (dict(d_k=0), 2), (dict(d_v=0), 2), (dict(dtype=2), 3), (dict(o_dtype=-1), 3), (dict(d_k=257), 4), (dict(d_v=300), 4),
           (dict(per_head=2), 4), (dict(q_stride_t=-1), 2), (dict(v_stride_b=-4), 2), (dict(a_stride_h=-1), 2),
           (dict(B=2 ** 20, H=2 ** 16, Hk=1, T=2 ** 20), 2)]
BAD_BLOCK = [(dict(B=0), 2), (dict(T=-1), 2), (dict(D=0), 2), (dict(dtype=7), 3), (dict(x_dtype=-1), 3), (dict(D=16385), 4),
             (dict(post=2), 4), (dict(act=3), 4), (dict(act=-1), 4), (dict(eps=0.0), 2), (dict(eps=float("nan")), 2),
             (dict(o_stride_t=-1), 2), (dict(x_stride_b=-1), 2), (dict(g_stride_t=-2), 2),
             (dict(B=2 ** 31 - 1, T=2 ** 31 - 1), 2)]


@pytest.mark.parametrize("entry,kw,status", [(e, kw, st) for e in CALLS for kw, st in (BAD_LIN if "lin" in e else BAD_BLOCK)])
def test_bad_shapes(lib_nogpu, entry, kw, status):  # noqa: F811
    if entry == "gdn_lin_step" and kw.get("T"):
        kw = {k: v for k, v in kw.items() if k != "T"} | {"B": 2 ** 31 - 1, "H": 2 ** 31 - 1, "Hq": 1, "Hk": 1}
    shape = CALLS[entry][0](**kw)
    first = CALLS[entry][2].split()[0]
    assert call(lib_nogpu, entry, shape, **{first: ODD}) == status
    assert lib_nogpu.gdn_last_error().decode() != ""
    if entry in WORKSPACE:
        assert getattr(lib_nogpu, entry + "_workspace_bytes")(ctypes.byref(shape)) == BIG


@pytest.mark.parametrize("entry", list(CALLS))
def test_missing_and_misaligned_arguments(lib_nogpu, entry):  # noqa: F811
    shape, names, required = CALLS[entry]
    assert call(lib_nogpu, entry, None) == 1
    for name in required.split():
        other = next(n for n in names.split() if n != name)
        assert call(lib_nogpu, entry, shape(), **{name: None, other: ODD}) == 1, name
    for name in names.split():
        assert call(lib_nogpu, entry, shape(), **{name: ODD}) == 4, name
        assert "aligned" in lib_nogpu.gdn_last_error().decode(), name
    if "step" in entry:
        assert call(lib_nogpu, entry, shape(T=2), q=ODD) == 2


def test_gradients_go_with_their_inputs(lib_nogpu):  # noqa: F811
    assert call(lib_nogpu, "gdn_lin_bwd", lin_shape(), log_alpha=None, q=ODD) == 1
    assert call(lib_nogpu, "gdn_block_norm_bwd", block_shape(), gate=None, o=ODD) == 1
    assert call(lib_nogpu, "gdn_block_norm_bwd", block_shape(), dgate=None, o=ODD) == 1
    assert call(lib_nogpu, "gdn_block_norm_bwd", block_shape(), dy=None, dx_out=None, o=ODD) == 1
    for name in ("w_post", "scale", "w_pre"):
        assert call(lib_nogpu, "gdn_block_norm_bwd", block_shape(), **{name: None}, o=ODD) == 1
    assert call(lib_nogpu, "gdn_block_norm_bwd", block_shape(), dy=None, o=ODD) == 1
    assert call(lib_nogpu, "gdn_block_norm_fwd", block_shape(), y=None, o=ODD) == 1
    assert call(lib_nogpu, "gdn_block_norm_fwd", block_shape(post=0), o=ODD) == 4
    assert "w_post" in lib_nogpu.gdn_last_error().decode()
    # in place needs a dense stream
    assert call(lib_nogpu, "gdn_block_norm_fwd", block_shape(x_stride_t=65)) == 4
    assert "contiguous" in lib_nogpu.gdn_last_error().decode()


@pytest.mark.parametrize("kw", [dict(T=2 ** 31 - 127, B=1, H=1, Hq=1, Hk=1), dict(T=2 ** 31 - 1, B=1, H=1, Hq=1, Hk=1)])
def test_tokens(lib_nogpu, kw):  # noqa: F811
    assert call(lib_nogpu, "gdn_lin_fwd", lin_shape(**kw), q=ODD) == 4
    assert "T must be at most" in lib_nogpu.gdn_last_error().decode()
    assert lib_nogpu.gdn_lin_fwd_workspace_bytes(ctypes.byref(lin_shape(**{**kw, "T": 2 ** 31 - 128}))) < BIG


@pytest.mark.parametrize("entry,kw", [("gdn_lin_fwd", dict(B=2 ** 22, T=1)), ("gdn_lin_bwd", dict(B=2 ** 21, T=1)),
                                      ("gdn_lin_bwd", dict(H=2 ** 22, Hq=2 ** 22, Hk=2 ** 22, B=1, T=1)),
                                      ("gdn_lin_bwd", dict(B=1, H=64, Hq=32, Hk=64, T=2 ** 22))])
def test_launch_limits(lib_nogpu, entry, kw):  # noqa: F811
    """More threads than a launch counts, refused by the query and the call."""
    shape = lin_shape(**kw)
    assert getattr(lib_nogpu, entry + "_workspace_bytes")(ctypes.byref(shape)) == BIG
    assert call(lib_nogpu, entry, shape, q=ODD) == 4
    assert "launch" in lib_nogpu.gdn_last_error().decode()


@pytest.mark.parametrize("entry", sorted(WORKSPACE))
def test_workspaces(lib_nogpu, entry):  # noqa: F811
    shape = CALLS[entry][0](T=4000)
    need = getattr(lib_nogpu, entry + "_workspace_bytes")(ctypes.byref(shape))
    assert 0 < need < BIG and need % 256 == 0
    good = ctypes.c_void_p(0x100000)
    other = {"x": ctypes.c_void_p(0x200000)}
    assert call(lib_nogpu, entry, shape, **other) == 5
    assert call(lib_nogpu, entry, shape, good, need - 1, **other) == 5
    assert call(lib_nogpu, entry, shape, ctypes.c_void_p(0x100010), need, **other) == 4


def test_segments_only_where_heads_are_few(lib_nogpu):  # noqa: F811
    query = lib_nogpu.gdn_lin_fwd_workspace_bytes
    many = lin_shape(B=4, H=16, Hq=16, Hk=16, d_k=128, d_v=128, T=4096)
    few = lin_shape(B=1, H=8, Hq=8, Hk=8, d_k=128, d_v=128, T=32768)
    short = lin_shape(B=1, H=8, Hq=8, Hk=8, d_k=128, d_v=128, T=256)
    assert query(ctypes.byref(many)) == 0 and query(ctypes.byref(short)) == 0
    # 16 segments of 2048 tokens: their states, and a decay each
    assert query(ctypes.byref(few)) == 8 * 16 * 128 * 128 * 4 + 8 * 16 * 4


def test_step_overlaps(lib_nogpu):  # noqa: F811
    """The state, or the output, in the memory of another operand."""
    entry, shape = "gdn_lin_step", lin_shape(B=3, T=1)
    size = {"q": (2 * 12800 + 64 + 64) * 2, "k": (2 * 25600 + 3 * 64 + 64) * 2, "v": (2 * 12800 + 3 * 32 + 32) * 2,
            "log_alpha": (2 * 400 + 3 + 1) * 4, "S": 3 * 4 * 32 * 64 * 4, "O": 3 * 4 * 32 * 2}
    for out in ("S", "O"):
        for other in size:
            if other == out or (out == "O" and other == "S"):
                continue
            base = {n: (i + 1) << 24 for i, n in enumerate(size)}
            for moved, to in ((out, base[other] + size[other] - 4), (other, base[out] + size[out] - 4)):
                ptrs = {n: ctypes.c_void_p(v) for n, v in {**base, moved: to}.items()}
                assert call(lib_nogpu, entry, shape, **ptrs) == 4, (out, other, moved)
                assert "overlap" in lib_nogpu.gdn_last_error().decode(), (out, other, moved)


def test_structs_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    types = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    for name, cls in (("gdn_lin_shape", _lib.GdnLinShape), ("gdn_block_norm_shape", _lib.GdnBlockNormShape)):
        end = text.index("} " + name + ";")
        body = text[text.rindex("typedef struct {", 0, end) + 16:end]
        want = [(w, types[line.replace(",", " ").split()[0]]) for line in body.split(";") if line.split()
                for w in line.replace(",", " ").split()[1:]]
        assert want == list(cls._fields_), name


# ---- the binding ----

@pytest.fixture
def here(monkeypatch, lib):  # noqa: F811
    """Calls on tensors of the "meta" device get as far as the library, which
    refuses their null pointers."""
    monkeypatch.setattr(_layer, "_elsewhere", lambda t, stream: False)
    monkeypatch.setattr(_layer, "_stream", lambda t: 0)
    monkeypatch.setattr(_layer, "_separate", lambda *a, **k: None)


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def lin_args(**kw):
    return {**dict(q=meta(2, 2, 9, 8), k=meta(2, 4, 9, 8), v=meta(2, 4, 9, 6), log_alpha=meta(2, 4, 9)), **kw}


@pytest.mark.parametrize("kw,error", [
    (dict(q=meta(2, 3, 9, 8)), ValueError), (dict(k=meta(2, 4, 9, 7)), ValueError), (dict(q=meta(2, 2, 8, 8)), ValueError),
    (dict(k=meta(2, 4, 9, 8, dtype=torch.bfloat16)), TypeError), (dict(v=meta(2, 4, 9, 6, dtype=torch.float16)), TypeError),
    (dict(v=meta(4, 9, 6)), ValueError), (dict(q=meta(2, 2, 8, 9).transpose(2, 3)), ValueError),
    (dict(log_alpha=meta(3)), ValueError), (dict(log_alpha=meta(2, 9, 4)), ValueError),
    (dict(log_alpha=meta(2, 4, 9, dtype=torch.bfloat16)), TypeError), (dict(S0=meta(2, 4, 8, 6)), ValueError),
    (dict(S0=meta(2, 4, 8, 6).transpose(2, 3)), ValueError), (dict(lens=meta(2)), TypeError),
    (dict(lens=meta(3, dtype=torch.int32)), ValueError)])
def test_binding_refuses(here, kw, error):
    with pytest.raises(gdn.GdnError):
        gdn.gdn_lin_fwd(**lin_args())                     # (null pointers)
    with pytest.raises(error):
        gdn.gdn_lin_fwd(**lin_args(**kw))
    with pytest.raises(error):
        gdn.gdn_lin_bwd(meta(2, 4, 9, 6, dtype=kw["v"].dtype if "v" in kw else torch.float32), **lin_args(**kw))


def test_binding_refuses_of_single_entries(here):
    a = lin_args()
    with pytest.raises(ValueError, match="dO"):
        gdn.gdn_lin_bwd(meta(2, 4, 6, 9).transpose(2, 3), **a)
    with pytest.raises(TypeError, match="dO"):
        gdn.gdn_lin_bwd(meta(2, 4, 9, 6, dtype=torch.bfloat16), **a)
    with pytest.raises(TypeError, match="O must"):
        gdn.gdn_lin_fwd(**a, o_dtype=torch.bfloat16, O=meta(2, 4, 9, 6))
    q, k, v = meta(2, 2, 8), meta(2, 4, 8), meta(2, 4, 6)
    with pytest.raises(ValueError, match="state"):
        gdn.gdn_lin_step(q, k, v)
    with pytest.raises(ValueError, match="S must"):
        gdn.gdn_lin_step(q, k, v, None, meta(2, 4, 8, 6))
    with pytest.raises(ValueError, match="log_alpha"):
        gdn.gdn_lin_step(q, k, v, meta(2, 4, 1), meta(2, 4, 6, 8))
    with pytest.raises(ValueError, match="divide"):
        gdn.gdn_lin_step(meta(2, 3, 8), k, v, None, meta(2, 4, 6, 8))


@pytest.mark.parametrize("kw,error", [
    (dict(x=meta(2, 9, 7)), ValueError), (dict(o=meta(2, 9, 8, dtype=torch.float16)), TypeError), (dict(w_pre=meta(7)), ValueError),
    (dict(scale=meta(1)), ValueError), (dict(gate=meta(2, 9, 8, dtype=torch.bfloat16)), TypeError), (dict(act="relu"), ValueError),
    (dict(post=False), ValueError), (dict(o=meta(9, 8)), ValueError), (dict(o=meta(2, 8, 9).transpose(1, 2)), ValueError)])
def test_binding_of_the_norms_refuses(here, kw, error):
    a = dict(o=meta(2, 9, 8), x=meta(2, 9, 8), w_pre=meta(8), w_post=meta(8), gate=meta(2, 9, 8), scale=meta(8))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_block_norm_fwd(**a)
    with pytest.raises(error):
        gdn.gdn_block_norm_fwd(**{**a, **kw})
    b = {**a, **kw}
    x = b.pop("x")
    with pytest.raises(error):
        gdn.gdn_block_norm_bwd(meta(2, 9, 8), meta(2, 9, 8), x, **b)


def test_binding_of_the_norms_refuses_halves(here):
    o, x, w = meta(2, 9, 8), meta(2, 9, 8), meta(8)
    with pytest.raises(ValueError, match="pre"):
        gdn.gdn_block_norm_fwd(o, x, w, pre=False)
    with pytest.raises(ValueError, match="dx_out or dy"):
        gdn.gdn_block_norm_bwd(None, None, x, o)
    with pytest.raises(ValueError, match="w_pre"):
        gdn.gdn_block_norm_bwd(meta(2, 9, 8), None, x, o, w)


@pytest.mark.parametrize("entry", ["lin_fwd", "lin_bwd", "lin_step", "block_norm_fwd", "block_norm_bwd"])
def test_dimensions_past_32_bits(here, entry):
    """A batch of 2^32 + 1 rows is not one of 1."""
    n = 2 ** 32 + 1
    big = lambda *s: meta(*s).expand(n, *s[1:])  # noqa: E731
    with pytest.raises(ValueError, match="below 2\\^31"):
        if entry == "lin_fwd":
            gdn.gdn_lin_fwd(big(1, 1, 1, 1), big(1, 1, 1, 1), big(1, 1, 1, 1))
        elif entry == "lin_bwd":
            gdn.gdn_lin_bwd(big(1, 1, 1, 1), big(1, 1, 1, 1), big(1, 1, 1, 1), big(1, 1, 1, 1))
        elif entry == "lin_step":
            gdn.gdn_lin_step(big(1, 1, 1), big(1, 1, 1), big(1, 1, 1), None, big(1, 1, 1, 1))
        elif entry == "block_norm_fwd":
            gdn.gdn_block_norm_fwd(big(1, 1, 1), big(1, 1, 1))
        else:
            gdn.gdn_block_norm_bwd(big(1, 1, 1), None, big(1, 1, 1), big(1, 1, 1))


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 1, 4, 8)
    for fn in (lambda: gdn.gdn_lin_fwd(x, x, x), lambda: gdn.gdn_lin_bwd(x, x, x, x),
               lambda: gdn.gdn_lin_step(x[0], x[0], x[0], None, torch.zeros(1, 4, 8, 8)),
               lambda: gdn.gdn_block_norm_fwd(x[0], x[0]), lambda: gdn.gdn_block_norm_bwd(x[0], x[0], x[0], x[0])):
        with pytest.raises(ValueError, match="GPU"):
            fn()


def test_every_name_is_exported():
    assert set(_mix.__all__) <= set(gdn.__all__) and all(callable(getattr(gdn, n)) for n in _mix.__all__)


def test_api_validation_under_asan_ubsan(tmp_path):
    """This file against a build whose host code of these entry points is
    instrumented (the device code is built as usual)."""
    if os.environ.get("GDN_TEST_LIB"):
        pytest.skip("already the instrumented run")
    from gated_delta_rule_13_amd import build as b
    rt = clang_asan_runtime()
    if rt is None or shutil.which(b.hipcc()) is None:
        pytest.skip("no clang sanitizer runtime in this ROCm")
    objs = [os.path.join(b.BUILD, u[0]) for u in b.units() if u[0] != "gdn_api_mix.o"]
    if not all(os.path.exists(o) for o in objs):
        b.build()
    api = str(tmp_path / "api.o")
    cmd = [b.hipcc(), f"--offload-arch={b.ARCH}", "-O1", "-g", "-std=c++17", "-fPIC", "-fno-omit-frame-pointer",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           f"-I{b.INCLUDE}", f"-I{b.CSRC}", "-c", os.path.join(b.CSRC, "gdn_api_mix.hip"), "-o", api]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    path = str(tmp_path / "libgdn_san.so")
    res = subprocess.run([b.hipcc(), f"--offload-arch={b.ARCH}", "-shared", "-fPIC", api, *objs, "-o", path],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    out = run_child(["-m", "pytest", "-q", "-p", "no:cacheprovider", "tests/test_mix_abi.py"],
                    {"LD_PRELOAD": rt, "GDN_TEST_LIB": path, "HIP_VISIBLE_DEVICES": "", "PYTHONPATH": ROOT})
    assert " passed" in out and " failed" not in out, out[-3000:]


# ---- the 64-bit references themselves ----

def test_reference_in_closed_form():
    """o_t = scale sum over i <= t of exp(G_t - G_i) (q_t . k_i) v_i, and what the
    first state leaves."""
    g = ref.gen(1)
    q, k, v = (ref.rand(g, 1, 2, 7, 5).double() for _ in range(3))
    la, S0 = -torch.rand(1, 2, 7, generator=g).double(), ref.rand(g, 1, 2, 5, 5).double()
    O, S = mix.lin(q, k, v, la, S0, scale=0.7)
    G = la.cumsum(-1)
    w = torch.exp(G[..., :, None] - G[..., None, :]).tril() * (q @ k.transpose(-1, -2))
    want = w @ v + torch.exp(G)[..., None] * (q @ S0.transpose(-1, -2))
    assert torch.allclose(O, 0.7 * want, atol=1e-12)
    short = mix.lin(q[:, :, :4], k[:, :, :4], v[:, :, :4], la[:, :, :4], S0)[1]
    assert torch.allclose(mix.lin(q, k, v, la, S0, lens=torch.tensor([4]))[1], short, atol=1e-13)


def test_reference_gradients_against_differences():
    g = ref.gen(2)
    a = {"q": ref.rand(g, 1, 1, 6, 4).double(), "k": ref.rand(g, 1, 2, 6, 4).double(), "v": ref.rand(g, 1, 2, 6, 3).double(),
         "log_alpha": -torch.rand(1, 2, 6, generator=g).double(), "S0": ref.rand(g, 1, 2, 3, 4).double()}
    cot = (ref.rand(g, 1, 2, 6, 3).double(), ref.rand(g, 1, 2, 3, 4).double())
    grads = ref.gradients(mix.lin, a, list(a), cot)
    for n in a:
        way = ref.rand(g, *a[n].shape).double()
        assert abs(float((grads[n] * way).sum()) - ref.difference(mix.lin, a, n, way, cot)) < 1e-6
    b = {"o": ref.rand(g, 1, 3, 5).double(), "x": ref.rand(g, 1, 3, 5).double(), "w_pre": ref.rand(g, 5).double(),
         "w_post": ref.rand(g, 5).double(), "gate": ref.rand(g, 1, 3, 5).double(), "scale": ref.rand(g, 5).double()}
    cot = (ref.rand(g, 1, 3, 5).double(), ref.rand(g, 1, 3, 5).double())
    grads = ref.gradients(mix.block, b, list(b), cot)
    for n in b:
        way = ref.rand(g, *b[n].shape).double()
        assert abs(float((grads[n] * way).sum()) - ref.difference(mix.block, b, n, way, cot)) < 1e-6
