"""The operators beside a compressed layer, made on one stream and used on another that was not told to wait."""
import contextlib

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
import adapter_reference as R

pytestmark = pytest.mark.gpu


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def keep_busy(d):
    """About 20 ms of ordinary work on the current stream."""
    a = torch.randn(8192, 8192, device=d).bfloat16()
    b = torch.empty_like(a)
    for _ in range(20):
        torch.mm(a, a, out=b)


@pytest.mark.parametrize("on_default", [True, False])
@pytest.mark.parametrize("given", [True, False])                  # the other stream: as an argument, or current
def test_a_plan_behind_other_work_is_waited_for(on_default, given):
    """The plan's memory holds the plan of another index before: results of that one would show."""
    d = dev()
    T, K, N, R_, L = 900, 128, 256, 8, 4
    g = torch.Generator().manual_seed(1)
    base, x, dy = ((torch.randn(T, w, generator=g)).bfloat16().to(d) for w in (N, K, N))
    down = (torch.randn(L, R_, K, generator=g) / K ** 0.5).bfloat16().to(d)
    up = (torch.randn(L, R_, N, generator=g) * 0.3).bfloat16().to(d)
    scaling = torch.ones(L, device=d)
    old, new = (torch.randint(-1, L, (T,), generator=g).int().to(d) for _ in range(2))
    memory = torch.empty(1 << 20, dtype=torch.uint8, device=d)
    want = R.adapters(base, x, None, down, up, scaling, new, None, dy, None)
    maker, side = torch.cuda.Stream(), torch.cuda.Stream()
    for grads in (False, True):
        E.AdapterPlan(old, L, workspace=memory)
        torch.cuda.synchronize()
        with contextlib.nullcontext() if on_default else torch.cuda.stream(maker):
            keep_busy(d)
            plan = E.AdapterPlan(new, L, workspace=memory)
        with contextlib.nullcontext() if given else torch.cuda.stream(side):
            stream = side if given else None
            if grads:
                got = E.adapter_grads(dy, x, down, up, scaling, plan, stream=stream)
            else:
                got = [E.adapter_add(base, x, down, up, scaling, plan, stream=stream)]
        torch.cuda.synchronize()
        for name, t in zip(("dx", "d_down", "d_up") if grads else ("out",), got):
            R.check(t, want[name], name)
