"""The middle of an expert layer keeps float32's 24 bits: sums that cancel but for their last bits, which are all exact."""
import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
import mxfp4_reference as R

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)


def stack(entries, n, rows, cols, four):
    """n copies of a matrix that is zero but for {(row, column): power of two}; at most one entry in 32 columns of a row."""
    v = torch.zeros(rows, cols)
    for (r, c), value in entries.items():
        v[r, c] = value
    if four:
        data, scales = R.store(*R.quantise(v))
        assert torch.equal(R.values(data, scales, cols), v.double())
        return E.MXFP4(data.to(D).expand(n, *data.shape).contiguous(), scales.to(D).expand(n, *scales.shape).contiguous(), cols)
    bytes_ = v.to(torch.float8_e4m3fn)
    assert torch.equal(bytes_.float(), v)
    return bytes_.view(torch.uint8).to(D).expand(n, rows, cols).contiguous()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T,n,top,one,K,inner", [(1, 4, 2, False, 96, 64), (6, 8, 1, True, 96, 288), (21, 16, 1, True, 608, 96), (16, 2, 2, False, 160, 544),
                                                 (40, 2, 1, False, 96, 160), (64, 300, 8, False, 128, 64), (60, 300, 1, True, 128, 1056)])
def test_the_last_bits_of_h_reach_the_result(T, n, top, one, K, inner, four, dtype):
    """h = 64 (1 + 2^-9 + 2^-s) in one place and 64 (1 + 2^-9) in another, whose difference, 2^(6 - s) for s from 19 to 23,
    is the result.  64 / (1 + exp(-64)) is 64 in float32."""
    p, q = inner - 1, 2
    gate = stack({(i, 0): 64.0 for i in range(inner)}, n, inner, K, four)
    up = stack({(p, 0): 1.0, (q, 0): 1.0, (p, 32): 2.0 ** -9, (q, 32): 2.0 ** -9, (p, 64): 2.0 ** -9}, n, inner, K, four)
    down = stack({**{(f, p): 1.0 for f in range(K)}, **{(f, q): -1.0 for f in range(K)}}, n, K, inner, four)
    x = torch.zeros(T, K)
    s = 19 + torch.arange(T) % 5
    x[:, 0], x[:, 32], x[:, 64] = 1.0, 1.0, 2.0 ** (9.0 - s)
    ids = torch.arange(T * top).reshape(T, top) % n if not one else torch.full((T, top), n - 1)
    y = E.moe_few(x.to(dtype).to(D), gate, up, down, ids.int().to(D), torch.ones(T, top, device=D))
    want = (top * 2.0 ** (6.0 - s))[:, None].expand(T, K)
    assert torch.equal(y.cpu().double(), want.double())
