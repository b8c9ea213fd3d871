"""What DecodePipeline.run hands to its layers with adapters, without a GPU: stand-ins for the plans, banks and layers."""
import types

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import adapters as A
from lossless_entropy_coded_ecf8_amd import pipeline as P


class Plan:
    made = []

    def __init__(self, index, adapters):
        self.adapters = adapters
        Plan.made.append(self)


class Layer:
    device = torch.device("cpu")

    def __init__(self, log):
        self.log = log

    def __call__(self, x, s, weight_u8=None, adapters=None, index=None):
        self.log.append(index if adapters is not None else None)
        return x


@pytest.fixture
def pipe(monkeypatch):
    log, Plan.made = [], []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(P, "AdapterPlan", Plan)

    def of(n):
        p = types.SimpleNamespace(layers=[Layer(log) for _ in range(n)], ahead=0, slots=1, slot=lambda i: None, log=log,
                                  plans=[types.SimpleNamespace(run=lambda s: None)] * n, _decode=lambda i, s: None, _check=lambda s: None)
        return p
    return of


def bank(rank, n=3):
    return types.SimpleNamespace(rank=rank, n_adapters=n, down=None)


def run(p, banks, index):
    n = len(banks)
    return E.DecodePipeline.run(p, [0] * n, [0] * n, adapters=banks, index=index)


def test_constants_are_the_headers():
    lib = A._lib()
    at = lambda t, r: lib.ecf8a_few(t, A.BankA(1, 1, 1, None, 64, 64, 1, r, 1, 0))  # noqa: E731
    assert at(A.FEW_TOKENS, A.FEW_RANK) == 1 and at(A.FEW_TOKENS + 1, 1) == 0 and at(1, A.FEW_RANK + 1) == 0


@pytest.mark.parametrize("tokens,ranks,plans", [(40, (8, 64), 0), (40, (100, 8, 100, 256), 1), (900, (8, 100, 16), 1)])
def test_an_index_is_grouped_once(pipe, tokens, ranks, plans):
    """Also for few tokens, where only ranks over 64 need it."""
    p, index = pipe(len(ranks) + 1), torch.zeros(tokens, dtype=torch.int32)
    run(p, [bank(r) for r in ranks] + [None], index)
    assert len(Plan.made) == plans and p.log[-1] is None
    for r, got in zip(ranks, p.log):
        assert got is (Plan.made[0] if tokens > 512 or r > 64 else index)


def test_banks_of_several_sizes_and_a_plan_given(pipe):
    p, index = pipe(3), torch.zeros(900, dtype=torch.int32)
    run(p, [bank(8, 3), bank(8, 5), bank(8, 3)], index)
    assert [q.adapters for q in Plan.made] == [3, 5] and [q.adapters for q in p.log] == [3, 5, 3]
    p = pipe(2)
    del p.log[:]
    given = Plan(index, 3)
    run(p, [bank(8), bank(100)], given)
    assert p.log == [given, given]
    with pytest.raises(ValueError):                               # before any layer has run
        run(p, [bank(8), bank(8, 4)], given)
    assert p.log == [given, given]
