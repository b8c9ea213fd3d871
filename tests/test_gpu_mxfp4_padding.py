"""What quantisation stores past the last value is zero, whatever the scale of E4M3 values is."""
import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
import mxfp4_reference as R

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)


@pytest.mark.parametrize("scale", [-0.5, float("nan"), float("inf"), -float("inf"), 0.0, -0.0])
@pytest.mark.parametrize("K", [32, 96, 160, 256])
def test_scales_of_any_sign_leave_the_padding_zero(K, scale):
    x = torch.randn(5, K, generator=torch.Generator().manual_seed(K)).to(torch.float8_e4m3fn)
    want = R.store(*R.quantise(x.float() * torch.tensor(scale)))
    q = E.quantize_mxfp4(x.to(D), torch.tensor(scale, device=D))
    assert torch.equal(q.scales.cpu(), want[1]) and torch.equal(q.data.cpu(), want[0])
    assert not bool(q.data[:, K // 2:].any()) and not bool(q.scales[:, K // 32:].any())
