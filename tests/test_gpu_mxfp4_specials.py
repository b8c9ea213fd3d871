"""Infinities, NaN and the ends of the scales' range in the products of 4-bit weights and in 4-bit experts."""
import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E
import mxfp4_reference as R

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)
BF, FP = torch.bfloat16, torch.float16


def gen(*seed):
    return torch.Generator().manual_seed(synth.seed_of("specials", *seed))


def check(got, ref, tol, what=""):
    """R.check, where infinities have to have their sign too."""
    R.check(got, ref, tol, what)
    at = torch.isinf(ref)
    assert torch.equal(got.detach().cpu().double()[at], ref[at]), what


def as_float16(ref):
    """What float16 makes of values that are past it: infinities of their sign."""
    return torch.where(ref.abs() >= 65520, torch.copysign(torch.full_like(ref, float("inf")), ref), ref)


@pytest.mark.parametrize("T,N,K", [(5, 40, 96), (70, 130, 288), (100, 1000, 544), (300, 64, 160)])
def test_input_grad_of_float16_under_the_largest_scales(T, N, K):
    """Blocks near 2^127 and 2^-127 beside ordinary ones: a dy of 0 stays 0, any other passes float16's range, with its sign."""
    g = gen(T, N, K)
    data, scales = R.random_stored((N,), K, g)
    data &= 0x77                                                  # no negative weights, so that no sum cancels
    data |= 0x22                                                  # and none is 0
    scales[:, : K // 32][torch.rand(N, K // 32, generator=g) < 0.3] = 254
    scales[:, : K // 32][torch.rand(N, K // 32, generator=g) < 0.2] = 0
    scales[:, 1] = torch.randint(0, 4, (N,), generator=g).to(torch.uint8)       # a block whose sums all vanish
    scales[:, 2] = torch.randint(250, 255, (N,), generator=g).to(torch.uint8)   # and one whose sums are all too large
    w, wv = E.MXFP4(data.to(D), scales.to(D), K), R.values(data, scales, K)
    dy = (torch.rand(T, N, generator=g) + 0.5).to(FP)
    dy[1::3] *= -1
    dy[2::5] = 0
    dy[4, 1:] = 0
    dy[4, 0] = 2.0 ** -24
    ref, tol = R.product(dy.double(), wv.t().contiguous(), FP)
    ref = as_float16(ref)
    assert bool(torch.isinf(ref).any()) and bool((ref[2::5] == 0).all())
    on = torch.zeros(T, N + -N % 8, dtype=FP, device=D)[:, :N]
    on.copy_(dy)
    check(E.linear_mxfp4_input_grad(on, w), ref, tol.nan_to_num(0.0, posinf=0.0), (T, N, K))


def test_input_grad_of_float16_whose_largest_terms_cancel():
    """Two weight rows of 6 2^127, past float32, that meet opposite signs: nothing is left, and of other columns what they have."""
    data, scales = torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.uint8)
    data[:2, :16], scales[:2, 0] = 0x77, 254                      # 32 codes of 6
    data[:, 16:32], scales[:, 1] = 0x22, 127                      # 32 codes of 1
    w = E.MXFP4(data.to(D), scales.to(D), 64)
    dy = torch.zeros(2, 8, dtype=FP, device=D)
    dy[0, :3] = torch.tensor([1.0, -1.0, 0.375])
    dy[1, :3] = torch.tensor([-2.0 ** -14, 2.0 ** -14, 5.0])
    dx = E.linear_mxfp4_input_grad(dy[:, :3], w).cpu()
    assert bool((dx[:, :32] == 0).all()) and torch.equal(dx[:, 32:], torch.tensor([[0.375], [5.0]], dtype=FP).expand(2, 32))
