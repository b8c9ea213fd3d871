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
