"""The 4-bit operators that keep no gradients say so, wherever a user's program may expect one."""
import warnings

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import mxfp4 as M


@pytest.mark.parametrize("name", ["quantize_mxfp4", "linear_mxfp4_input_grad"])
def test_a_call_that_keeps_no_gradients_says_so_once(name, monkeypatch):
    """Off the GPU, where every call is refused after that."""
    monkeypatch.setattr(M, "_warned", set())
    w = E.MXFP4(torch.zeros(5, 64, dtype=torch.uint8), torch.zeros(5, 4, dtype=torch.uint8), 64)
    call = {"quantize_mxfp4": lambda x: E.quantize_mxfp4(x), "linear_mxfp4_input_grad": lambda x: E.linear_mxfp4_input_grad(x, w)}[name]

    def heard(x):
        with warnings.catch_warnings(record=True) as got:
            warnings.simplefilter("always")
            with pytest.raises(ValueError):
                call(x)
        assert all(str(m.message).startswith(name + " keeps no gradients") for m in got)
        return len(got)

    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    leaf = x.clone().requires_grad_()
    with torch.no_grad():
        assert heard(leaf) == 0
    assert [heard(x), heard(leaf), heard(leaf)] == [0, 1, 0]
    monkeypatch.setattr(M, "_warned", set())
    if name == "quantize_mxfp4":                                  # the scale of E4M3 values may carry one too
        call = lambda s: E.quantize_mxfp4(x.to(torch.float8_e4m3fn), s)      # noqa: E731
        assert heard(torch.ones((), requires_grad=True)) == 1


@pytest.mark.parametrize("which", ["x", "weights", "gate_scale", "up_scale", "down_scale"])
def test_every_operand_of_an_expert_layer_is_looked_at(which, monkeypatch):
    monkeypatch.setattr(M, "_warned", set())
    u8 = torch.zeros(2, 32, 32, dtype=torch.uint8)
    given = dict(x=torch.zeros(3, 32, dtype=torch.bfloat16), weights=torch.zeros(3, 1), gate_scale=torch.ones(2), up_scale=torch.ones(2), down_scale=torch.ones(2))
    given[which].requires_grad_()
    with warnings.catch_warnings(record=True) as got:
        warnings.simplefilter("always")
        with pytest.raises(ValueError):
            E.moe_few(gate=u8, up=u8, down=u8, ids=torch.zeros(3, 1, dtype=torch.int32), **given)
    assert len(got) == 1 and "moe_few" in str(got[0].message)
