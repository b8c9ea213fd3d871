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
