"""The bounds that linear attention's GPU tests hold outputs to reject what they
are there for: results that are off by a per cent, gradients of a decay without
the pairs around a chunk, operands rounded once more (on the CPU, with the exact
results in the kernels' place)."""
import pytest
import torch

from tests import layer_ref as ref
from tests import mix_ref as mix
from tests.test_lin_decay_gpu import reference, row
from tests.test_lin_gpu import BF, F32, SCALE, inputs
from tests.test_lin_rounding_gpu import once


def rejected(name, got, want, bound):
    with pytest.raises(AssertionError, match=name):
        once(name, got, want, bound)


@pytest.mark.parametrize("T,dk,dv,strong", [(400, 64, 64, 0.02), (300, 32, 96, 0.1)])
def test_decays(T, dk, dv, strong):
    a, dO = row(BF, T, dk, dv, T, strong)
    want, bound = reference(a, dO, None)
    once("dlog_alpha", want.float(), want, bound)
    rejected("dlog_alpha", (want * 1.01).float(), want, bound)
    # the second chunk of 64 without the pairs around it: without what is written
    # before it, read behind it
    w = ref.wide(a)
    first, last = (torch.zeros(1, 1, T, 1, dtype=torch.float64) for _ in range(2))
    first[:, :, :64], last[:, :, 128:] = 1, 1
    cut, _ = reference({**w, "v": w["v"] * first}, dO.double() * last, None)
    less = want.clone()
    less[:, :, 64:128] -= cut[:, :, 64:128]
    rejected("dlog_alpha", less.float(), want, bound)


def test_documents_do_not_take_each_other_s_rounding():
    """2^-20 of the second document's gradient added to the first's."""
    a, dO = row(BF, 300, 32, 32, 1)
    a["log_alpha"][..., 150] = -float("inf")
    dO[:, :, :150] *= 2.0 ** -17
    want, bound = reference(a, dO, None)
    once("dlog_alpha", want.float(), want, bound)
    more = want.clone()
    more[:, :, :150] += 2.0 ** -20 * want[:, :, 150:].abs().max()
    rejected("dlog_alpha", more.float(), want, bound)


@pytest.mark.parametrize("name", ["O", "dq", "dk", "dv"])
def test_outputs_in_bf16(name):
    """Of exact inputs: rounded once it passes; from rows rounded once more, or off
    by a per cent, it does not."""
    a = inputs(1, 2, 2, 2, 200, 64, 64, F32, 4)
    w = ref.wide(a)
    dO = ref.rand(ref.gen(1), 1, 2, 200, 64).double()
    other = {"O": "k", "dq": "k", "dk": "q", "dv": "q"}[name]

    def value(x, do, absolute=False):
        if absolute:
            x, do = {n: v if n in ("log_alpha", "lens") or v is None else v.abs() for n, v in x.items()}, do.abs()
        if name == "O":
            return mix.lin(**x, scale=SCALE)[0]
        return ref.gradients(lambda **k: mix.lin(**k, scale=SCALE), x, [name[1:]], (do, None))[name[1:]]
    want, bound = value(w, dO), value(w, dO, True)
    once(name, want.to(BF), want, bound)
    rejected(name, (want * 1.01).to(BF), want, bound)
    coarse = {**w, other: w[other].to(BF).double()}
    rejected(name, value(coarse, dO).to(BF), want, bound)
