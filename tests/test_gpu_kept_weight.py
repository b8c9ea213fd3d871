"""ECF8Linear.adapted with a decoded weight that the caller keeps for the backward pass."""
import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E

pytestmark = pytest.mark.gpu


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def setup(d, n=3):
    layers = [E.ECF8Linear(torch.from_numpy(synth.small_stable(128 * 128, 1.8, i)).view(128, 128), scale=2e-4, device=d) for i in range(n)]
    bank = E.AdapterBank(2, 4, 128, 128, device=d)
    g = torch.Generator().manual_seed(3)
    with torch.no_grad():
        bank.up.copy_((torch.randn(2, 4, 128, generator=g) * 0.1).bfloat16())
    x = torch.randn(40, 128, generator=g).bfloat16().to(d).requires_grad_(True)
    index = (torch.arange(40, device=d) % 2).int()
    return layers, bank, x, index


def gradient(y, x):
    return torch.autograd.grad(y, [x], torch.ones_like(y))[0]


def test_a_kept_weight_that_torch_writes_is_refused():
    d = dev()
    layers, bank, x, index = setup(d)
    w = layers[0].decoded_weight().clone()
    want = gradient(layers[0].adapted(x, bank, index), x)
    y = layers[0].adapted(x, bank, index, weight_u8=w)
    assert torch.equal(gradient(y, x), want)
    y = layers[0].adapted(x, bank, index, weight_u8=w)
    w.copy_(layers[1].decoded_weight())
    with pytest.raises(RuntimeError):
        gradient(y, x)


@pytest.mark.parametrize("slots,ahead", [(3, 2), (2, 1), (1, 0)])
def test_a_slot_that_takes_another_layer_is_refused(slots, ahead):
    """... and one that is decoded again for the same layer, or lies beside, is not."""
    d = dev()
    layers, bank, x, index = setup(d)
    xs = [torch.zeros(16, 128, device=d).to(torch.float8_e4m3fn)] * 3
    ss = [torch.ones((), device=d)] * 3
    pipe = E.DecodePipeline(layers, slots=slots, ahead=ahead)
    pipe.run(xs, ss)
    for i in range(3 - slots, 3):                                  # the layers that the slots hold now
        want = gradient(layers[i].adapted(x, bank, index), x)
        y = layers[i].adapted(x, bank, index, weight_u8=pipe.slot(i))
        assert torch.equal(gradient(y, x), want)
        y = layers[i].adapted(x, bank, index, weight_u8=pipe.slot(i))
        pipe.run(xs, ss)
        if not any(j != i and j % slots == i % slots for j in range(3)):   # no other layer's slot: the same bytes again
            assert torch.equal(gradient(y, x), want)
        else:
            with pytest.raises(RuntimeError):
                gradient(y, x)


def test_weights_that_stay_are_taken():
    """The layer's own buffer, decoded again in between, and one made in inference mode."""
    d = dev()
    layers, bank, x, index = setup(d, 1)
    want = gradient(layers[0].adapted(x, bank, index), x)
    y = layers[0].adapted(x, bank, index, weight_u8=layers[0].decoded_weight())
    layers[0].decoded_weight()
    assert torch.equal(gradient(y, x), want)
    with torch.inference_mode():
        w = layers[0].decoded_weight().clone()
    assert w.is_inference()
    assert torch.equal(gradient(layers[0].adapted(x, bank, index, weight_u8=w), x), want)


def test_a_layer_that_comes_twice():
    """Its slot is decoded again at the second place: the same bytes."""
    d = dev()
    layers, bank, x, index = setup(d, 1)
    xs, ss = [torch.zeros(16, 128, device=d).to(torch.float8_e4m3fn)] * 2, [torch.ones((), device=d)] * 2
    pipe = E.DecodePipeline([layers[0]] * 2, slots=1, ahead=0)
    pipe.run(xs, ss)
    y = layers[0].adapted(x, bank, index, weight_u8=pipe.slot(1))
    pipe.run(xs, ss)
    assert torch.equal(gradient(y, x), gradient(layers[0].adapted(x, bank, index), x))
