"""Microscaled 4-bit weights on the GPU: conversion bit for bit, products and the input gradient against float64."""
import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E
import mxfp4_reference as R

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)
BF, FP, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def gen(*seed):
    return torch.Generator().manual_seed(synth.seed_of(*seed))


def as_mx(data, scales, K):
    return E.MXFP4(data.to(D), scales.to(D), K)


def weight(N, K, seed, lo=110, hi=128):
    data, scales = R.random_stored((N,), K, gen("w", N, K, seed), lo, hi)
    return as_mx(data, scales, K), R.values(data, scales, K)


def spread(t, pad, lead=0):
    """t as columns of a wider buffer, which is filled with NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device=t.device).to(t.dtype)
    view = wide[:, lead:lead + t.shape[1]]
    view.copy_(t)
    return view


# ------------------------------------------------------------------ conversion

@pytest.mark.parametrize("dtype", [BF, FP, F32, F8])
@pytest.mark.parametrize("rows,K,pad,lead", [(1, 32, 0, 0), (1, 128, 0, 0), (3, 96, 0, 0), (5, 160, 8, 0), (7, 4096, 0, 0), (33, 544, 3, 1),
                                             (257, 1024, 16, 16), (2, 32768, 0, 0)])
def test_quantise_bit_for_bit(dtype, rows, K, pad, lead):
    g = gen(rows, K, pad)
    v = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-20, 8, (rows, K // 32), generator=g)).repeat_interleave(32, 1)
    if dtype == F8:
        v = v.clamp(-448, 448)
    x = v.to(dtype)
    scale = torch.tensor(0.037) if dtype == F8 else None
    f = x.float() * scale if dtype == F8 else x.float()
    want = R.store(*R.quantise(f))
    on = x.to(D)
    on = spread(on, pad, lead) if pad else on
    q = E.quantize_mxfp4(on, None if scale is None else scale.to(D))
    assert q.shape == (rows, K) and q.features == K
    assert torch.equal(q.scales.cpu(), want[1])
    assert torch.equal(q.data.cpu(), want[0])
    assert torch.equal(q.dequantize(F32).cpu().double(), R.values(*want, K))


@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_quantise_ties_signs_and_ends_of_the_range(dtype):
    """Every tie and its neighbours under several scales; zeros of both signs; the largest and smallest numbers of the
    type; infinities and NaN, alone in their block."""
    info = torch.finfo(dtype)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375, 0.0, 0.5, 1.0, 2.0, 3.0, 4.0])
    rows = []
    for e in (-14, -3, 0, 2, 5, 12):
        m = torch.cat([ties, -ties]) * 2.0 ** e
        rows += [m, m * (1 + 2.0 ** -7), m * (1 - 2.0 ** -7)]
    rows += [torch.zeros(32), -torch.zeros(32), torch.full((32,), info.max), torch.full((32,), -info.max),
             torch.full((32,), info.tiny), torch.full((32,), info.smallest_normal / 8), torch.linspace(-1, 1, 32) * info.tiny]
    for bad in (float("inf"), -float("inf"), float("nan")):
        for at in (0, 13, 31):
            r = torch.ones(32)
            r[at] = bad
            rows.append(r)
    x = torch.stack(rows).to(dtype)
    want = R.store(*R.quantise(x.float()))
    q = E.quantize_mxfp4(x.to(D))
    assert torch.equal(q.scales.cpu(), want[1])
    assert torch.equal(q.data.cpu(), want[0])
    back = q.dequantize(F32).cpu().double()
    assert torch.equal(torch.isnan(back), torch.isnan(R.values(*want, 32)))


def test_quantise_smallest_float32_numbers():
    """A block whose scale is held at 2^-127: its values are rounded to steps of half of that."""
    x = torch.linspace(-1, 1, 32 * 8).reshape(8, 32) * torch.exp2(torch.arange(-133.0, -117.0, 2.0, dtype=torch.float64))[:, None]
    x = x.float()
    want = R.store(*R.quantise(x))
    q = E.quantize_mxfp4(x.to(D))
    assert torch.equal(q.scales.cpu(), want[1]) and torch.equal(q.data.cpu(), want[0])


def test_dequantise_every_code_under_every_scale():
    code = torch.arange(16, dtype=torch.uint8).repeat(2).expand(256, 32).contiguous()
    data, scales = R.store(code, torch.arange(256, dtype=torch.uint8)[:, None].contiguous())
    want = R.values(data, scales, 32)
    for dtype in (F32, BF, FP):
        got = as_mx(data, scales, 32).dequantize(dtype).cpu()
        ref = want.to(F32).to(dtype)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got.nan_to_num(7.0), ref.nan_to_num(7.0)), dtype
        assert torch.equal(torch.signbit(got[:255]), torch.signbit(ref[:255])), dtype


def test_quantise_stack_and_out_and_stream():
    x = torch.randn(3, 5, 96, generator=gen(1)).bfloat16()
    want = R.store(*R.quantise(x.float().reshape(15, 96)))
    q = E.quantize_mxfp4(x.to(D))
    assert q.shape == (3, 5, 96) and torch.equal(q.data.cpu().reshape(15, -1), want[0])
    out = E.MXFP4(torch.full_like(q.data, 0xAB), torch.full_like(q.scales, 0xCD), 96)
    side = torch.cuda.Stream()
    on = x.to(D)
    side.wait_stream(torch.cuda.current_stream())
    assert E.quantize_mxfp4(on, out=out, stream=side) is out
    y = out.dequantize(BF, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.data, q.data) and torch.equal(out.scales, q.scales) and torch.equal(y, q.dequantize(BF))


def test_quantise_past_32_bits():
    rows, K = 140000, 32768                                       # 4.6e9 bytes of E4M3
    x = torch.zeros(rows, K, dtype=torch.uint8, device=D)
    part = torch.randint(0, 256, (3, K), generator=gen(2)).to(torch.uint8)
    part[(part & 127) == 127] = 5                                 # no NaN
    at = [0, 131072, rows - 1]
    x[at] = part.to(D)
    q = E.quantize_mxfp4(x.view(F8))
    want = R.store(*R.quantise(part.view(F8).float()))
    assert torch.equal(q.data[at].cpu(), want[0]) and torch.equal(q.scales[at].cpu(), want[1])
    back = q.dequantize(BF)
    assert torch.equal(back[at].cpu().double(), R.values(*want, K))
    assert int(q.data.view(torch.int64).count_nonzero()) == int(q.data[at].contiguous().view(torch.int64).count_nonzero())


# ------------------------------------------------------------------ products

SIZES = [(1, 1, 32), (1, 17, 4096), (1, 256, 8224), (2, 33, 96), (7, 130, 128), (16, 100, 160), (17, 64, 544), (31, 5, 1024), (32, 300, 320),
         (33, 129, 576), (64, 257, 608), (65, 256, 64), (66, 3, 128), (100, 131, 224), (128, 256, 512), (130, 515, 2080), (257, 260, 96),
         (300, 1030, 352), (513, 769, 288), (90, 40, 8192)]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "mx", "mx_fp16"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear_against_float64(T, N, K, kind):
    g = gen(T, N, K)
    dtype = FP if "fp16" in kind else BF
    w, wv = weight(N, K, 1)
    x = (torch.randn(T, K, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dtype)
    for with_bias in (False, True):
        b = (torch.randn(N, generator=g) * 4).to(dtype) if with_bias else None
        shift = None if b is None else b.double()
        on_b = None if b is None else b.to(D)
        if kind.startswith("mx"):
            stored = R.store(*R.quantise(x.float()))
            ref, tol = R.product(R.values(*stored, K), wv, dtype, shift)
            got = E.linear_mxfp4(as_mx(*stored, K), w, on_b, out_dtype=dtype)
        else:
            ref, tol = R.product(x.double(), wv, dtype, shift)
            got = E.linear_mxfp4(x.to(D), w, on_b)
        assert got.dtype == dtype
        R.check(got, ref, tol, (kind, T, N, K, with_bias))


@pytest.mark.parametrize("T", [1, 20, 200])
def test_linear_slices_leave_the_rest_alone(T):
    N, K = 100, 224
    w, wv = weight(N, K, 2)
    x = torch.randn(T, K, generator=gen(T)).bfloat16()
    on = spread(x.to(D), 24, 8)
    ref, tol = R.product(x.double(), wv, BF)
    for lead, pad in ((0, 4), (3, 9), (8, 8)):
        wide = torch.full((T + 2, N + pad + lead), 77.0, dtype=BF, device=D)
        out = wide[1:T + 1, lead:lead + N]
        assert E.linear_mxfp4(on, w, out=out) is out
        R.check(out, ref, tol, (lead, pad))
        wide[1:T + 1, lead:lead + N] = 77.0
        assert bool((wide == 77.0).all())


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_linear_keeps_infinities_and_nan_in_their_rows(T, dtype):
    """A row of x with an infinity or NaN, and a weight row with a NaN block: as the formula has them, and nowhere else."""
    N, K = 70, 288
    data, scales = R.random_stored((N,), K, gen(5))
    data |= 0x11                                                  # no zero weights: an infinity stays one
    data[:, K // 2:] = 0
    scales[9, 2] = 255
    w, wv = as_mx(data, scales, K), R.values(data, scales, K)
    x = torch.randn(T, K, generator=gen(6)).to(dtype)
    x[1, 7], x[2, 3] = float("inf"), float("nan")
    ref, tol = R.product(x.double(), wv, dtype)
    # a sum that holds an infinity is that infinity; tolerances of such rows say nothing
    got = E.linear_mxfp4(x.to(D), w)
    R.check(got, ref, tol.nan_to_num(0.0, posinf=0.0))


@pytest.mark.parametrize("T", [2, 100])
def test_linear_extreme_scales(T):
    """Weights near 2^-107 and 2^97, and blocks that float16 could not hold beside each other under float16 activations."""
    x = torch.randn(T, 160, generator=gen(T)) * 1e-2
    for lo, hi, dtype in ((20, 22, BF), (224, 226, BF), (80, 128, FP)):
        w, wv = weight(48, 160, lo, lo, hi)
        v = x.to(dtype)
        R.check(E.linear_mxfp4(v.to(D), w), *R.product(v.double(), wv, dtype), (T, lo))


def test_linear_past_32_bits():
    N, K = (1 << 20), 8224                                        # 4.4e9 bytes of codes
    data = torch.zeros(N, 8320 // 2, dtype=torch.uint8, device=D)
    scales = torch.zeros(N, 8320 // 32, dtype=torch.uint8, device=D)
    at = [0, 1, 524289, N - 2, N - 1]
    part = R.random_stored((len(at),), K, gen(7))
    data[at], scales[at] = part[0].to(D), part[1].to(D)
    w = E.MXFP4(data, scales, K)
    for T in (1, 70):
        x = torch.randn(T, K, generator=gen(T)).bfloat16()
        y = E.linear_mxfp4(x.to(D), w)
        ref, tol = R.product(x.double(), R.values(*part, K), BF)
        R.check(y[:, at], ref, tol, T)
        assert int(y.count_nonzero()) <= T * len(at)


# ------------------------------------------------------------------ input gradient

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 40, 4096), (3, 64, 96), (16, 65, 128), (33, 130, 288), (64, 1000, 256), (65, 63, 544),
                                   (129, 128, 512), (200, 77, 1056), (257, 320, 800), (300, 1111, 224), (40, 8192, 64), (513, 192, 608)])
def test_input_grad_against_float64(T, N, K, dtype):
    g = gen(T, N, K)
    w, wv = weight(N, K, 3)
    dy = (torch.randn(T, N, generator=g) * 0.1).to(dtype)
    ref, tol = R.product(dy.double(), wv.t().contiguous(), dtype)
    on = spread(dy.to(D), -N % 8 + 8, 8)                          # rows on 16-byte borders, NaN around them
    R.check(E.linear_mxfp4_input_grad(on, w), ref, tol, (T, N, K))


def test_input_grad_out_and_nan():
    T, N, K = 70, 200, 160
    data, scales = R.random_stored((N,), K, gen(8))
    scales[3, 1] = 255
    w, wv = as_mx(data, scales, K), R.values(data, scales, K)
    dy = torch.randn(T, N, generator=gen(9)).bfloat16()
    dy[5, 6] = float("nan")
    ref, tol = R.product(dy.double(), wv.t().contiguous(), BF)
    wide = torch.full((T + 1, K + 16), 5.0, dtype=BF, device=D)
    out = wide[:T, 8:8 + K]
    assert E.linear_mxfp4_input_grad(dy.to(D), w, out=out) is out
    R.check(out, ref, tol.nan_to_num(0.0))
    wide[:T, 8:8 + K] = 5.0
    assert bool((wide == 5.0).all())


def test_input_grad_is_the_derivative_of_the_product():
    """Differences of the product along random directions, in float64 of the kernels' float32-exact weights."""
    w, wv = weight(96, 256, 11)
    dy = torch.randn(5, 96, generator=gen(1)).bfloat16()
    dx = E.linear_mxfp4_input_grad(dy.to(D), w).cpu().double()
    x, v = torch.randn(5, 256, generator=gen(2)).double(), torch.randn(5, 256, generator=gen(3)).double()
    f = lambda z: float(((z @ wv.t()) * dy.double()).sum())       # noqa: E731
    slope = (f(x + 1e-3 * v) - f(x - 1e-3 * v)) / 2e-3
    # each dx value is rounded to bfloat16: 2^-8 of its magnitude
    assert abs(slope - float((dx * v).sum())) <= 2.0 ** -8 * float((dx.abs() * v.abs()).sum()) * 1.01 + 1e-9 * abs(slope)


# ------------------------------------------------------------------ streams, graphs, determinism

def test_captured_products_replay_as_they_ran():
    w, _ = weight(300, 512, 4)
    xs = {T: torch.randn(T, 512, generator=gen(T)).bfloat16().to(D) for T in (3, 90)}
    dy = torch.randn(90, 304, generator=gen(5)).bfloat16().to(D)[:, :300]

    def step():
        return [E.linear_mxfp4(xs[3], w), E.linear_mxfp4(xs[90], w), E.linear_mxfp4(E.quantize_mxfp4(xs[90]), w),
                E.linear_mxfp4_input_grad(dy, w), E.quantize_mxfp4(xs[90]).dequantize(BF)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        for x in xs.values():
            x.copy_(torch.randn(x.shape, generator=gen(i, x.shape[0])).bfloat16())
        dy.copy_(torch.randn(dy.shape, generator=gen(i, 1)).bfloat16())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_two_streams_at_once_give_the_same_bits():
    w, _ = weight(700, 2048, 6)
    x = torch.randn(80, 2048, generator=gen(8)).bfloat16().to(D)
    dy = torch.randn(80, 704, generator=gen(9)).bfloat16().to(D)[:, :700]
    want = E.linear_mxfp4(x, w), E.linear_mxfp4_input_grad(dy, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in streams:
            got.append((E.linear_mxfp4(x, w, stream=s), E.linear_mxfp4_input_grad(dy, w, stream=s)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_no_tokens():
    w, _ = weight(20, 64, 1)
    assert E.linear_mxfp4(torch.empty(0, 64, dtype=BF, device=D), w).shape == (0, 20)
    assert E.linear_mxfp4_input_grad(torch.empty(0, 24, dtype=BF, device=D)[:, :20], w).shape == (0, 64)
    q = E.quantize_mxfp4(torch.empty(0, 64, dtype=BF, device=D))
    assert q.shape == (0, 64) and q.dequantize().shape == (0, 64) and E.linear_mxfp4(q, w).shape == (0, 20)
