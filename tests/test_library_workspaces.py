"""Workspaces of the adapters' gradients follow what a batch can need (sizes only: no GPU)."""
import ctypes
import random

import pytest

from lossless_entropy_coded_ecf8_amd import adapters as A


def plan_of(tokens, adapters):
    """The bounds that ecf8a_plan_prepare fills in (it needs a GPU): see include/ecf8a.h."""
    unit = max(256, (((tokens + 15) // 16) + 63) // 64 * 64)
    bare, used = min(adapters + 1, tokens), min(adapters, tokens)
    return A.PlanA(1 << 40, 1 << 40, tokens, adapters, (tokens + 15 * bare) // 16 * 16, tokens // 64 + bare, tokens // unit + used, unit)


def grads_bytes(tokens, adapters, rank, k, n):
    bank = A.BankA(1 << 40, 1 << 40, 1 << 40, None, k, n, adapters, rank, 1, 0)
    return A._lib().ecf8a_grads_bytes(ctypes.byref(plan_of(tokens, adapters)), ctypes.byref(bank))


def test_gradients_of_a_large_bank():
    """8192 tokens of a bank of 2048 adapters: at most 32 units (of 512 slots) belong to adapters that have several."""
    assert grads_bytes(8192, 2048, 64, 8192, 8192) < 1 << 30
    forms = 3 * 4 * plan_of(8192, 2048).max_slots * 64
    assert grads_bytes(8192, 2048, 64, 8192, 8192) >= forms + 32 * 64 * 2 * 8192 * 4
    assert grads_bytes(200, 2048, 64, 8192, 8192) < 1 << 28        # fewer tokens than one unit: no sums at all


@pytest.mark.parametrize("seed", range(20))
def test_partial_sums_of_any_index_fit(seed):
    """The room for partial sums, read from how the workspace grows with the width, against the units of adapters with
    several, for banks used evenly, by a few, and each just past one unit."""
    rng = random.Random(seed)
    adapters, tokens = rng.choice([1, 2, 7, 40, 500, 2048]), rng.choice([1, 255, 256, 257, 511, 513, 4096, 4097, 8192, 70001])
    p = plan_of(tokens, adapters)
    # the widths share every other part of the workspace: wide enough for one share, a multiple of 128
    per = 4 * 16 * 128 * 512                                     # bytes of one unit's sums at rank 16 over 512 strips
    wide, wider = (grads_bytes(tokens, adapters, 16, w * 128, 128) for w in (512, 1024))
    room = (wider - wide) / per
    counts = {"even": [tokens // adapters + (a < tokens % adapters) for a in range(adapters)]}
    few = [0] * adapters
    for _ in range(tokens):
        few[min(int(rng.expovariate(0.3)), adapters - 1)] += 1
    counts["few"] = few
    past, left = [], tokens
    while left and len(past) < adapters:
        past.append(min(left, p.unit_slots + 1))
        left -= past[-1]
    counts["past"] = past
    for kind, c in counts.items():
        units = [-(-(-(-n // 16) * 16) // p.unit_slots) for n in c]
        assert sum(u for u in units if u > 1) <= room, (kind, tokens, adapters)
