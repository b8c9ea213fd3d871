"""DecodePipeline.run with banks of several ranks and sizes."""
import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [16, 48, 700])
def test_banks_of_several_ranks_and_sizes(tokens):
    """Bit for bit what each layer gives by itself."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    d = torch.device("cuda", 0)
    layers = [E.ECF8Linear(torch.from_numpy(synth.small_stable(256 * 128, 1.8, i)).view(256, 128), scale=2e-4, device=d) for i in range(4)]
    banks = [E.AdapterBank(n, r, 128, 256, device=d) if r else None for n, r in ((3, 100), (3, 8), (2, 72), (0, 0))]
    g = torch.Generator().manual_seed(tokens)
    with torch.no_grad():
        for b in banks[:3]:
            b.up.copy_((torch.randn(b.up.shape, generator=g) * 0.1).bfloat16())
    xs = [(torch.randn(tokens, 128, generator=g) * 4).to(torch.float8_e4m3fn).to(d) for _ in layers]
    ss = [torch.tensor(0.25, device=d)] * 4
    index = torch.randint(-1, 3, (tokens,), generator=g).int().to(d)
    pipe = E.DecodePipeline(layers, slots=2, ahead=1)
    for ix in (index, index.long()):
        for i, got in enumerate(pipe.run(xs, ss, adapters=banks, index=ix)):
            assert torch.equal(got, layers[i](xs[i], ss[i], adapters=banks[i], index=ix)), i
    with pytest.raises(ValueError):
        pipe.run(xs, ss, adapters=banks, index=E.AdapterPlan(index, 3))
