"""The factors' gradients of banks where some adapters have several units of tokens and others one."""
import ctypes

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import adapters as A
import adapter_reference as R
from test_gpu_adapters import dev, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,L,tokens_each", [(8192, 2048, 513), (5000, 30, 321), (9000, 9, 2000), (300, 3, 257)])
def test_adapters_of_one_unit_and_of_several(T, L, tokens_each, dtype):
    """Partial sums have room for every unit of an adapter with several, and nothing is written past the workspace."""
    d = dev()
    s = make(d, T, 40, 24, 5, L, "tokens", dtype, seed=L)
    many = torch.arange(T, device=d) // tokens_each * 2 + 1       # every second adapter: just past a unit
    s["index"] = torch.where(many < L, many, s["index"].long()).int()
    s["index"] = s["index"][torch.randperm(T, generator=torch.Generator().manual_seed(T)).to(d)].contiguous()
    plan = E.AdapterPlan(s["index"], L)
    bank = A._bank(s["down"], s["up"], s["scaling"], None, d)
    need = A._lib().ecf8a_grads_bytes(ctypes.byref(plan.c), ctypes.byref(bank))
    memory = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=d)
    got = E.adapter_grads(s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan, dx_base=s["dx_base"], workspace=memory[:need])
    want = reference(s, True)
    for name, t in zip(("dx", "d_down", "d_up"), got):
        R.check(t, want[name], name)
    assert bool((memory[need:] == 0x5A).all())
