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


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [1, 4, 16, 40, 64, 65, 150, 400])
@pytest.mark.parametrize("N,K", [(70, 288), (300, 1056)])
def test_infinities_in_activations_keep_their_sign(T, N, K, dtype):
    """A sum that meets one infinity is that infinity times its weight's sign, one that meets two of opposite signs NaN; other rows are as ever."""
    g = gen(T, N, K)
    data, scales = R.random_stored((N,), K, g)
    data[:, : K // 2] |= 0x11                                     # no zero weights
    w, wv = E.MXFP4(data.to(D), scales.to(D), K), R.values(data, scales, K)
    x = torch.randn(T, K, generator=g).to(dtype)
    inf = float("inf")
    x[0, 7] = inf
    x[T // 2, K - 1] = -inf
    x[T - 1, 3], x[T - 1, 70] = inf, -inf
    ref, tol = R.product(x.double(), wv, dtype)
    assert bool((ref == inf).any()) and bool((ref == -inf).any())
    check(E.linear_mxfp4(x.to(D), w), ref, tol.nan_to_num(0.0, posinf=0.0), (T, N, K))


@pytest.mark.parametrize("T", [1, 4, 16, 40, 64, 65, 150, 400])
@pytest.mark.parametrize("N,K", [(70, 288), (300, 1056), (9, 96)])
def test_blocks_of_nan_in_either_operand_of_a_four_bit_product(T, N, K):
    g = gen(T, N, K, 1)
    data, scales = R.random_stored((N,), K, g)
    scales[N // 2, 1], scales[N - 1, K // 32 - 1] = 255, 255
    w, wv = E.MXFP4(data.to(D), scales.to(D), K), R.values(data, scales, K)
    xd, xs = R.random_stored((T,), K, g)
    if T > 2:
        xs[1, 0], xs[T - 1, K // 32 - 1] = 255, 255
    xv = R.values(xd, xs, K)
    for dtype in (BF, FP):
        ref, tol = R.product(xv, wv, dtype)
        ref = as_float16(ref) if dtype == FP else ref
        got = E.linear_mxfp4(E.MXFP4(xd.to(D), xs.to(D), K), w, out_dtype=dtype)
        check(got, ref, tol.nan_to_num(0.0, posinf=0.0), (T, N, K, dtype))
        assert bool(torch.isnan(ref[:, N // 2]).all()) and (T <= 2 or bool(torch.isnan(ref[1]).all()))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,N,K", [(1, 40, 96), (20, 130, 160), (70, 200, 160), (100, 1000, 544), (300, 72, 288)])
def test_infinities_and_nan_in_the_gradient_of_the_output(T, N, K, dtype):
    g = gen(T, N, K, 2)
    data, scales = R.random_stored((N,), K, g)
    data[:, : K // 2] |= 0x11
    scales[5, 1] = 255                                            # a NaN block: one 32 columns of every row
    w, wv = E.MXFP4(data.to(D), scales.to(D), K), R.values(data, scales, K)
    dy = torch.randn(T, N, generator=g).to(dtype)
    inf = float("inf")
    dy[0, 3] = inf
    if T > 3:
        dy[1, N - 1], dy[2, 0], dy[2, 9], dy[3, 4] = -inf, inf, -inf, float("nan")
    ref, tol = R.product(dy.double(), wv.t().contiguous(), dtype)
    on = torch.zeros(T, N + -N % 8, dtype=dtype, device=D)[:, :N]
    on.copy_(dy)
    check(E.linear_mxfp4_input_grad(on, w), ref, tol.nan_to_num(0.0, posinf=0.0), (T, N, K))


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("T,n,top", [(1, 4, 2), (12, 4, 2), (40, 2, 1), (64, 300, 4)])
def test_blocks_of_nan_in_four_bit_experts(T, n, top, which):
    """gate, up or down of one expert: its tokens' results are NaN, in every feature (gate, up) or the block's row, and no other's."""
    g = gen(T, n, top, which)
    given, values = [], []
    for m, (rows, cols) in enumerate(((96, 128), (96, 128), (128, 96))):
        data, scales = R.random_stored((n, rows), cols, g, 117, 123)
        if m == which:
            scales[1, 17, 2] = 255
        given.append(E.MXFP4(data.to(D), scales.to(D), cols))
        values.append(R.values(data, scales, cols))
    x = torch.randn(T, 128, generator=g).bfloat16()
    ids = torch.randint(0, n, (T, top), generator=g).int()
    ids[0, 0] = 1
    w = torch.rand(T, top, generator=g) + 0.5
    ref, tol = R.layer(x.double(), *values, ids, w.double(), BF)
    bad = (ids == 1).any(1)
    assert torch.equal(torch.isnan(ref).any(1), bad) and (which == 2 or bool(torch.isnan(ref[bad]).all()))
    check(E.moe_few(x.to(D), *given, ids.to(D), w.to(D)), ref, tol.nan_to_num(0.0), (T, n, top))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,n,top", [(1, 4, 2), (7, 4, 1), (40, 2, 1), (64, 300, 4)])
@pytest.mark.parametrize("four", [False, True])
def test_results_of_experts_past_the_types_range_have_their_sign(T, n, top, four, dtype):
    """h past bfloat16's range, an infinity of x, and results past float16's: as float32 sums have them, rounded."""
    g = gen(T, n, top, four, 3)
    given, values = [], []
    for rows, cols in ((32, 64), (32, 64), (64, 32)):
        if four:
            data, scales = R.random_stored((n, rows), cols, g, 124, 128)
            data &= 0x77                                          # no negative weights, none of 0
            data |= 0x22
            given.append(E.MXFP4(data.to(D), scales.to(D), cols))
            values.append(R.values(data, scales, cols))
        else:
            b = (torch.rand(n, rows, cols, generator=g) + 0.5).to(torch.float8_e4m3fn)
            given.append(b.view(torch.uint8).to(D))
            values.append(b.double())
    x = torch.rand(T, 64, generator=g).to(dtype) + 1
    x[0, 5] = float("inf")
    if T > 2:
        x[2] = x[2] * 2.0 ** (70 if dtype == BF else 14)          # the product of gate and up is past float32
    ids = torch.randint(0, n, (T, top), generator=g).int()
    w = -torch.ones(T, top)
    ref, tol = R.layer(x.double(), *values, ids, w.double(), dtype)
    most = 3.38e38 if dtype == BF else 65520
    if dtype == BF and T > 2:
        assert bool((ref[2] < -3.5e38).all())
    ref = torch.where(ref.abs() >= most, torch.copysign(torch.full_like(ref, float("inf")), ref), ref)
    check(E.moe_few(x.to(D), *given, ids.to(D), w.to(D)), ref, tol.nan_to_num(0.0, posinf=0.0), (T, n, top))


@pytest.mark.parametrize("T", [1, 4, 16, 40, 64, 65, 150, 400])
@pytest.mark.parametrize("N,K", [(70, 288), (300, 1056)])
def test_products_under_the_largest_and_smallest_scales(T, N, K):
    """float16 activations, and both operands in 4 bits: zeros stay zeros, what passes the type's range has its sign, what is too small vanishes."""
    g = gen(T, N, K, 4)
    data, scales = R.random_stored((N,), K, g)
    data &= 0x77                                                  # no negative weights, so that no sum cancels
    data |= 0x22
    kind = torch.randint(0, 3, (N, 1), generator=g)
    scales[:, : K // 32] = torch.where(kind == 0, 254, torch.where(kind == 1, 0, scales[:, : K // 32])).to(torch.uint8)
    w, wv = E.MXFP4(data.to(D), scales.to(D), K), R.values(data, scales, K)
    x = (torch.rand(T, K, generator=g) + 0.5).to(FP)
    x[::3] *= -1
    if T > 1:
        x[1::4] = 0
    ref, tol = R.product(x.double(), wv, FP)
    check(E.linear_mxfp4(x.to(D), w), as_float16(ref), tol.nan_to_num(0.0, posinf=0.0), (T, N, K))
    xd, xs = R.random_stored((T,), K, g)
    xd = (xd & 0x77) | 0x22
    sign = torch.randint(0, 2, (T, 1), generator=g).to(torch.uint8)
    xd |= sign * 0x88
    xs[:, : K // 32] = torch.where(torch.randint(0, 2, (T, 1), generator=g) == 0, 254, 0).to(torch.uint8)
    if T > 1:
        xd[1::4] = 0
    ref, tol = R.product(R.values(xd, xs, K), wv, BF)
    ref = torch.where(ref.abs() >= 3.4e38, torch.copysign(torch.full_like(ref, float("inf")), ref), ref)
    got = E.linear_mxfp4(E.MXFP4(xd.to(D), xs.to(D), K), w)
    check(got, ref, torch.where(torch.isinf(ref), 0.0, tol), (T, N, K))
