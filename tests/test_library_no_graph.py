"""Entry points that keep no gradients say so, once, where an operand requires them (no GPU: the call itself is refused)."""
import warnings

import pytest
import torch

from lossless_entropy_coded_ecf8_amd import adapters as A


def operands(grad):
    down, up = torch.zeros(1, 2, 4, dtype=torch.bfloat16), torch.zeros(1, 2, 4, dtype=torch.bfloat16)
    return dict(base=None, x=torch.zeros(3, 4, dtype=torch.bfloat16), down=down.requires_grad_(grad), up=up, scaling=torch.ones(1),
                index=torch.zeros(3, dtype=torch.int32))


@pytest.fixture(autouse=True)
def fresh(monkeypatch):
    monkeypatch.setattr(A, "_warned", False)


def heard(call):
    with warnings.catch_warnings(record=True) as got:
        warnings.simplefilter("always")
        call()
    return [str(w.message) for w in got]


def add(grad):
    with pytest.raises(ValueError):                               # the index is not on a GPU
        A.adapter_add(**operands(grad))


def test_adapter_add_says_that_no_gradient_is_kept():
    assert heard(lambda: add(False)) == []
    with torch.no_grad():
        assert heard(lambda: add(True)) == []
    got = heard(lambda: add(True))
    assert len(got) == 1 and "adapted" in got[0]
    assert heard(lambda: add(True)) == []                         # once


def test_a_bank_says_so_too(monkeypatch):
    monkeypatch.setattr(A, "adapter_add", lambda y, *a, **k: y)
    bank, y = A.AdapterBank(1, 2, 4, 4, device="cpu"), torch.zeros(3, 4)
    with torch.inference_mode():
        assert heard(lambda: bank.add_(y, y, None)) == []
    assert len(heard(lambda: bank.add_(y, y, None))) == 1
    monkeypatch.setattr(A, "_warned", False)
    bank.requires_grad_(False)
    assert heard(lambda: bank.add_(y, y, None)) == []
