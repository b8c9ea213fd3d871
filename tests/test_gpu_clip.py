"""The global norm of many gradients and their clipping, against the formula in 64 bits."""
import math

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-44}


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def grads_of(sizes, dtype, d, seed=0, scale=1.0, shift=False):
    g = torch.Generator().manual_seed(seed)
    got = []
    for i, n in enumerate(sizes):
        off = (i * 3 + 1) % 8 if shift else 0
        buf = torch.full((n + off + 9,), float("nan")).to(dtype).to(d)
        buf[off:off + n] = (torch.randn(n, generator=g) * scale).to(dtype).to(d)
        got.append(buf[off:off + n])
    return got


def check(before, after, norm, max_norm):
    """The norm is one float32 rounding (and one of the square root's last place) off; a scaled value one rounding of
    the factor to float32 and one product's, then its type's."""
    flat = [g.float().cpu().double() for g in before]
    want = math.sqrt(math.fsum(float((f * f).sum()) for f in flat))
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    c = min(1.0, max_norm / (want + 1e-6))
    for f, a in zip(flat, after):
        dt = a.dtype
        ref = f * c
        tol = ref.abs() * (HALF[dt] + 2.0 ** -22) * (1 + 2.0 ** -6) + TINY[dt]
        assert bool(((a.float().cpu().double() - ref).abs() <= tol).all())


SIZES = [[1], [7], [8, 0, 3], [4096], [5, 300, 4099, 70000], [0, 0], [65536] * 3 + [1] * 40, [2 ** 20 + 3, 17],
         [1 << 22, 999, 1 << 19]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%d" % sum(s))
@pytest.mark.parametrize("shift", [False, True])
def test_clip_against_formula(sizes, dtype, shift):
    d = dev()
    grads = grads_of(sizes, dtype, d, seed=len(sizes), scale=0.1, shift=shift)
    before = [g.clone() for g in grads]
    for max_norm in (0.05, 1e9):
        out = [torch.zeros(g.numel() + 3, dtype=dtype, device=d)[3 if i % 2 else 0:][:g.numel()] for i, g in enumerate(grads)]
        norm = E.clip_grad_norm(grads, max_norm, out=out)
        for g, b in zip(grads, before):
            assert torch.equal(g, b)
        check(before, out, norm, max_norm)
    norm = E.clip_grad_norm(grads, 0.05)
    check(before, grads, norm, 0.05)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_not_finite_and_large(dtype):
    """An infinity makes the factor 0, a NaN makes everything NaN; squares past float32 do not overflow."""
    d = dev()
    big = {torch.bfloat16: 1e30, torch.float16: 6e4, torch.float32: 1e30}[dtype]
    g = [torch.full((5000,), big, dtype=dtype, device=d), torch.ones(7, dtype=dtype, device=d)]
    out = [torch.empty_like(t) for t in g]
    norm = E.clip_grad_norm(g, 1.0, out=out)
    want = math.sqrt(5000 * float(g[0][0]) ** 2 + 7)
    assert abs(float(norm) / want - 1) < 2.0 ** -23
    check(g, out, norm, 1.0)
    g[1][3] = float("inf")
    norm = E.clip_grad_norm(g, 1.0, out=out)
    assert float(norm) == float("inf") and bool((out[0] == 0).all())
    assert bool(torch.isnan(out[1][3])) and bool((out[1][:3] == 0).all())
    g[0][100] = float("nan")
    norm = E.clip_grad_norm(g, 1.0, out=out)
    assert bool(torch.isnan(norm)) and all(bool(torch.isnan(o).all()) for o in out)


def test_plan_follows_the_values_and_replays():
    """A plan reads the gradients anew each run, on any stream, captured or not; what lies beside them is not touched."""
    d = dev()
    grads = grads_of([100, 70001, 3, 5000], torch.bfloat16, d, scale=0.01, shift=True)
    out = [torch.empty_like(g) for g in grads]
    plan = E.GradClip(grads, out=out)
    in_place = E.GradClip(grads)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = plan.run(0.5)
    for k in range(1, 5):
        for g in grads:
            g.mul_(1.5)
        before = [g.clone() for g in grads]
        graph.replay()
        torch.cuda.synchronize()
        check(before, out, held, 0.5)
        first = [o.clone() for o in out]
        norm = plan.run(0.5)
        torch.cuda.synchronize()
        assert torch.equal(norm, held) and all(torch.equal(a, b) for a, b in zip(first, out))
        st.wait_stream(torch.cuda.current_stream())
        norm = plan.run(0.5, stream=st)
        st.synchronize()
        assert torch.equal(norm, held)
    norm = in_place.run(1e9)                                      # a factor of 1: nothing is written
    check(before, grads, norm, 1e9)
    norm = in_place.run(0.5)
    check(before, grads, norm, 0.5)


def test_refusals():
    d = dev()
    a = torch.ones(64, device=d)
    for grads, out in (([], None), ([a, a], None), ([a, a[10:20]], None), ([a, a.half()], None), ([a.double()], None),
                       ([a.cpu()], None), ([a[::2]], None), ([a], [a[:63]]), ([a[:32]], [a[16:48]]), ([a], [a, a]),
                       ([a[:8], a[8:16]], [a[8:16], a[:8]])):
        with pytest.raises((ValueError, E.Ecf8Error)):
            E.clip_grad_norm(grads, 1.0, out=out)
    for bad in (-1.0, float("nan")):
        with pytest.raises(E.Ecf8Error):
            E.clip_grad_norm([a], bad)
    assert float(E.clip_grad_norm([a], float("inf"))) == 8.0 and bool((a == 1).all())
    E.clip_grad_norm([a], 0.0)
    assert bool((a == 0).all())
