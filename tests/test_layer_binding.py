"""Argument checks of the binding of the operators around the recurrence, on
tensors without memory."""
import pytest
import torch

import gated_delta_rule_13_amd as gdn
from gated_delta_rule_13_amd import _layer
from tests.test_abi import lib  # noqa: F401


@pytest.fixture
def here(monkeypatch, lib):  # noqa: F811
    """Calls on tensors of the "meta" device get as far as the library, which
    refuses their null pointers."""
    monkeypatch.setattr(_layer, "_elsewhere", lambda t, stream: False)
    monkeypatch.setattr(_layer, "_stream", lambda t: 0)
    monkeypatch.setattr(_layer, "_separate", lambda *a, **k: None)      # (all at address 0)


def meta(*shape, of=None, dtype=torch.float32):
    """A tensor of a shape, or a broadcast one of another shape."""
    t = torch.empty(shape, dtype=dtype, device="meta")
    return t if of is None else t.expand(of)


CALLS = {
    "gdn_conv_fwd": lambda x: gdn.gdn_conv_fwd(x(1, 1, 1), meta(1, 4)),
    "gdn_conv_bwd": lambda x: gdn.gdn_conv_bwd(meta(1, 1, 1), x(1, 1, 1), meta(1, 4)),
    "gdn_conv_step": lambda x: gdn.gdn_conv_step(x(1, 1), meta(1, 4), None, meta(1, 3, 1)),
    "gdn_ssm_fwd": lambda x: gdn.gdn_ssm_fwd(x(1, 1, 1), x(1, 1, 1), meta(1, 1), meta(1, 1, 1, 1), meta(1, 1, 1, 1)),
    "gdn_ssm_bwd": lambda x: gdn.gdn_ssm_bwd(meta(1, 1, 1), x(1, 1, 1), x(1, 1, 1), meta(1, 1), meta(1, 1, 1, 1),
                                             meta(1, 1, 1, 1)),
    "gdn_ssm_step": lambda x: gdn.gdn_ssm_step(x(1, 1), x(1, 1), meta(1, 1), meta(1, 1, 1), meta(1, 1, 1), h=meta(1, 1, 1)),
    "gdn_norm_fwd": lambda x: gdn.gdn_norm_fwd(x(1, 1, 1, 1)),
    "gdn_norm_bwd": lambda x: gdn.gdn_norm_bwd(meta(1, 1, 1, 1), x(1, 1, 1, 1)),
}


@pytest.mark.parametrize("entry", sorted(CALLS))
def test_dimensions_past_32_bits(here, entry):
    """A batch of 2^32 + 1 rows is not one of 1."""
    with pytest.raises(gdn.GdnError):                 # (a shape that is fine, and null pointers)
        CALLS[entry](lambda *s: meta(*s))
    with pytest.raises(ValueError, match="below 2\\^31"):
        CALLS[entry](lambda *s: meta(*s, of=(2 ** 32 + 1,) + s[1:]))
