"""The operators beside a compressed layer, made on one stream and used on another that was not told to wait."""
import contextlib
import ctypes
import math

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import adapters as A
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


def test_a_clip_refused_in_a_capture_leaves_the_capture_whole():
    """A GradClip made inside a capture is refused, by the library too; one made before runs in it."""
    d = dev()
    grads = [torch.randn(n, device=d) for n in (1000, 7, 70000)]
    before = [g.clone() for g in grads]
    plan = E.GradClip(grads, out=[torch.empty_like(g) for g in grads])
    arr, c = (A.GradA * 1)(A.GradA(grads[0].data_ptr(), grads[0].data_ptr(), 1000)), A.ClipPlanA()
    memory = torch.zeros(1 << 16, dtype=torch.uint8, device=d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError):
            E.GradClip(grads)
        with pytest.raises(RuntimeError):
            E.clip_grad_norm(grads, 1.0)
        rc = A._lib().ecf8a_clip_prepare(arr, 1, 3, memory.data_ptr(), memory.numel(), torch.cuda.current_stream().cuda_stream,
                                         ctypes.byref(c))
        norm = plan.run(0.5)
    assert rc == -1 and c.pieces == 0
    want = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in before))
    for _ in range(3):
        for o in plan.out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        # one float32 rounding of the norm and one of its root; a scaled value: the factor's rounding, then its own
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
        for g, b, o in zip(grads, before, plan.out):
            ref = b.double() * (0.5 / (want + 1e-6))
            assert torch.equal(g, b) and bool(((o.double() - ref).abs() <= ref.abs() * 2.0 ** -22 + 1e-44).all())
    assert bool((memory == 0).all())


def test_runs_of_one_clip_on_two_streams():
    """Run after run on alternating streams, each with a larger norm allowed: all see one norm, and what stands at the end
    is the last run's."""
    d = dev()
    grads = [torch.randn(1 << 20, device=d) for _ in range(8)]
    out = [torch.empty_like(g) for g in grads]
    plan = E.GradClip(grads, out=out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    norms, first = [], [g.clone() for g in grads]
    torch.cuda.synchronize()
    for k in range(8):
        norms.append(plan.run(1e-3 * (k + 1), stream=streams[k % 2]))
    torch.cuda.synchronize()
    want = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in first))
    for n in norms:
        assert abs(float(n) - want) <= 2.0 ** -23 * want
    for g, o in zip(first, out):
        ref = g.double() * (8e-3 / (want + 1e-6))
        # 8e-3 is rounded to float32, as are the factor and the product
        assert bool(((o.double() - ref).abs() <= ref.abs() * (2.0 ** -22 + 2.0 ** -24) + 1e-44).all())
