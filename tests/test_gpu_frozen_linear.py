"""The gradient a frozen E4M3 weight passes to its input, against the formula in 64 bits."""
import math

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
import adapter_reference as R

pytestmark = pytest.mark.gpu


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def e4m3_table():
    """The value of each byte from its bits: bias 7, subnormals at 2^-9 a step, 0x7F and 0xFF NaN."""
    got = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        got.append(math.nan if b & 127 == 127 else -v if b & 128 else v)
    return torch.tensor(got, dtype=torch.float64)


def reference(dy, w, scale):
    """Exact products, N float32 additions (N 2^-23 of the magnitudes), one scaling (2^-23), one rounding."""
    dy, w, scale = dy.float().cpu().double(), e4m3_table()[w.cpu().long()], float(scale)
    ref = dy @ w * scale
    err = (dy.abs() @ w.abs()) * abs(scale) * (w.shape[0] + 8) * 2.0 ** -23
    return ref, err


def make(T, N, K, dtype, d, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(T, N + pad, generator=g).to(dtype).to(d)[:, :N]
    w = torch.randint(0, 256, (N, K), generator=g, dtype=torch.uint8)
    w[(w & 127) == 127] = 0x70
    return dy, w.to(d), torch.tensor(2.0 ** -7 * 0.83, device=d)


SIZES = [(1, 16, 16), (1, 4096, 256), (2, 48, 32), (17, 16, 144), (31, 80, 400), (64, 512, 128), (100, 1040, 272),
         (33, 4112, 48), (2048, 144, 6160),
         (127, 64, 1040), (129, 112, 128), (200, 3088, 64), (257, 256, 528), (513, 336, 656), (1025, 64, 1296)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_input_grad_against_formula(size, dtype):
    d = dev()
    T, N, K = size
    dy, w, s = make(T, N, K, dtype, d, seed=T + N)
    ref, err = reference(dy, w, s)
    R.check(E.linear_fp8_input_grad(dy, w, s), (ref, R.rounded(ref, err, dtype)), size)


def test_rounds_once_for_every_e4m3_byte():
    """One token, one-hot rows: dx is w_scale times each byte's value, rounded once; NaN bytes give NaN."""
    d = dev()
    w = torch.arange(256, dtype=torch.uint8).repeat(16, 1)
    for i in range(16):
        w[i] = torch.roll(w[i], i)
    table = e4m3_table()
    s = torch.tensor(0.75, device=d)
    for dtype in (torch.bfloat16, torch.float16):
        dy = torch.eye(16, dtype=dtype, device=d)
        clean = torch.where((w & 127) == 127, torch.zeros_like(w), w)
        got = E.linear_fp8_input_grad(dy, clean.to(d), s).cpu()
        assert torch.equal(got, (table[clean.long()] * 0.75).to(dtype))
        got = E.linear_fp8_input_grad(dy, w.to(d), s).cpu()          # a NaN anywhere in a column makes all of it NaN
        assert torch.equal(torch.isnan(got), torch.isnan(table[w.long()]).any(0, keepdim=True).expand(16, 256))


def test_infinities_and_nan_keep_to_their_rows():
    d = dev()
    for T, N, K in ((40, 80, 64), (300, 1104, 400)):
        dy, w, s = make(T, N, K, torch.bfloat16, d, seed=5)
        w = (w & 0x3F) + 1                                        # positive, not 0
        want = E.linear_fp8_input_grad(dy, w, s)
        dy[3, N - 1] = float("nan")
        dy[7, 2] = float("-inf")
        dy[9, N - 2] = float("inf")
        got = E.linear_fp8_input_grad(dy, w, s)
        keep = torch.ones(T, dtype=torch.bool, device=d)
        keep[[3, 7, 9]] = False
        assert torch.equal(got[keep], want[keep]) and bool(torch.isnan(got[3]).all())
        assert bool((got[7] == float("-inf")).all()) and bool((got[9] == float("inf")).all())


def test_slices_streams_and_replays():
    """Rows of wider buffers, what lies beside them untouched; another stream; captured and replayed."""
    d = dev()
    T, N, K = 70, 2080, 336
    dy, w, s = make(T, N, K, torch.bfloat16, d, seed=6, pad=24)
    want = E.linear_fp8_input_grad(dy.contiguous(), w, s)
    buf = torch.full((T + 2, K + 40), 3.0, dtype=torch.bfloat16, device=d)
    out = E.linear_fp8_input_grad(dy, w, s, out=buf[1:T + 1, 16:16 + K])
    assert torch.equal(out, want)
    edge = buf.clone()
    edge[1:T + 1, 16:16 + K] = 3.0
    assert bool((edge == 3.0).all())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = E.linear_fp8_input_grad(dy, w, s, stream=st)
    st.synchronize()
    assert torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    x = dy.contiguous()
    with torch.cuda.graph(g):
        o = E.linear_fp8_input_grad(x, w, s)
    for k in range(4):
        x.copy_(dy * (k + 1))
        g.replay()
        eager = E.linear_fp8_input_grad(x, w, s)
        torch.cuda.synchronize()
        assert torch.equal(o, eager)


def test_more_than_two_to_the_31_elements():
    d = dev()
    T, N, K = 70000, 16, 32768
    g = torch.Generator().manual_seed(1)
    dy = torch.randn(T, N, generator=g).bfloat16().to(d)
    w = torch.randint(0, 0x70, (N, K), generator=g, dtype=torch.uint8).to(d)
    s = torch.tensor(0.01, device=d)
    out = E.linear_fp8_input_grad(dy, w, s)
    for rows in (slice(0, 3), slice(T - 3, T)):
        ref, err = reference(dy[rows], w, s)
        R.check(out[rows], (ref, R.rounded(ref, err, torch.bfloat16)))
    del out
    torch.cuda.empty_cache()


def test_one_row_of_any_stride():
    d = dev()
    dy, w, s = make(1, 96, 64, torch.bfloat16, d, seed=8)
    want = E.linear_fp8_input_grad(dy, w, s)
    for stride in (1, 97, 1 << 24):
        assert torch.equal(E.linear_fp8_input_grad(dy.as_strided((1, 96), (stride, 1)), w, s), want)


def test_refusals():
    d = dev()
    dy, w, s = make(8, 48, 64, torch.bfloat16, d)
    E.linear_fp8_input_grad(dy, w, s)
    assert E.linear_fp8_input_grad(dy[:0], w, s).shape == (0, 64)
    odd = torch.empty(8, 49, dtype=torch.bfloat16, device=d)
    for args in ((dy.float(), w, s), (dy, w.float(), s), (dy[:, :47], w, s), (dy, w.t(), s), (dy, w, s.double()), (dy.cpu(), w, s),
                 (dy[0], w, s), (dy, w[:, :63].contiguous(), s), (odd[:, :48], w, s), (odd[:, 1:], w, s),
                 (torch.empty(8, 40, dtype=torch.bfloat16, device=d), w[:40].contiguous(), s)):
        with pytest.raises((ValueError, E.Ecf8Error)):
            E.linear_fp8_input_grad(*args)
    with pytest.raises(ValueError):
        E.linear_fp8_input_grad(dy, torch.zeros(48, 48, dtype=torch.uint8, device=d), s, out=dy)
