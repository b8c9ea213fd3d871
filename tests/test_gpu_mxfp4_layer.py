"""A 4-bit layer as it is used: beside a compressed one, serving with adapters, trained with adapters."""
import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E
import adapter_reference as A
import mxfp4_reference as R

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)
BF, FP, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def gen(*seed):
    return torch.Generator().manual_seed(synth.seed_of(*seed))


def compressed(out, inn, seed, bias=True):
    w = torch.from_numpy(synth.small_stable(out * inn, 1.8, seed)).view(out, inn)
    b = torch.randn(out, generator=gen(seed)).bfloat16() if bias else None
    return w, E.ECF8Linear(w, scale=2e-3, bias=b, device=D)


def bank_of(layer, n, rank, dtype=BF, ranks=None):
    g = gen(n, rank)
    bank = E.AdapterBank(n, rank, layer.in_features, layer.out_features, scaling=torch.linspace(0.5, 1.5, n), ranks=ranks, dtype=dtype, device=D)
    with torch.no_grad():
        bank.down.copy_((torch.randn(bank.down.shape, generator=g) / layer.in_features ** 0.5).to(dtype))
        bank.up.copy_((torch.randn(bank.up.shape, generator=g) * 0.1).to(dtype))
    return bank


def test_four_bit_form_of_a_compressed_layer():
    w, full = compressed(200, 256, 1)
    layer = E.MXFP4Linear.from_ecf8(full)
    stored = R.store(*R.quantise(w.view(F8).float() * torch.tensor(2e-3)))
    assert torch.equal(layer.weight.data.cpu(), stored[0]) and torch.equal(layer.weight.scales.cpu(), stored[1])
    wv, b = R.values(*stored, 256), full.bias.cpu().double()
    for T in (1, 30, 100):
        x = torch.randn(T, 256, generator=gen(T)).bfloat16()
        R.check(layer(x.to(D)), *R.product(x.double(), wv, BF, b))
        layer.four_bit_input = True
        xv = R.values(*R.store(*R.quantise(x.float())), 256)
        R.check(layer(x.to(D)), *R.product(xv, wv, BF, b))
        layer.four_bit_input = False
    lin = torch.nn.Linear(64, 24)
    small = E.MXFP4Linear.from_linear(lin, device=D)
    want = R.store(*R.quantise(lin.weight.detach()))
    assert torch.equal(small.weight.data.cpu(), want[0]) and small.bias.dtype == torch.float32
    x = torch.randn(3, 64, generator=gen(4)).to(FP)
    R.check(small(x.to(D)), *R.product(x.double(), R.values(*want, 64), FP, lin.bias.detach().to(FP).double()))
    state = small.state_dict()
    assert set(state) == {"data", "scales", "bias"}
    again = E.MXFP4Linear.from_linear(torch.nn.Linear(64, 24), device=D)
    again.load_state_dict(state)
    assert torch.equal(again(x.to(D)), small(x.to(D)))


@pytest.mark.parametrize("T", [1, 50, 600])
def test_serving_with_adapters(T):
    _, full = compressed(320, 512, 2)
    layer = E.MXFP4Linear.from_ecf8(full)
    bank = bank_of(layer, 4, 12, ranks=[12, 3, 0, 7])
    x = torch.randn(T, 512, generator=gen(T)).bfloat16().to(D)
    index = torch.randint(-1, 4, (T,), generator=gen(T, 1)).int().to(D)
    base = layer(x)
    want = A.adapters(base, x, None, bank.down, bank.up, bank.scaling, index, bank.ranks)["out"]
    with torch.no_grad():
        A.check(layer(x, adapters=bank, index=index), want)
    with pytest.raises(ValueError):
        layer(x, adapters=bank)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,out", [(5, 272), (130, 273), (800, 272)])
def test_training_against_formula(T, out, dtype):
    _, full = compressed(out, 384, 3)
    layer = E.MXFP4Linear.from_ecf8(full)
    bank = bank_of(layer, 3, 10, dtype, ranks=[10, 4, 9])
    g = gen(T)
    x = torch.randn(T, 384, generator=g).to(dtype).to(D).requires_grad_(True)
    dy = (torch.randn(T, out, generator=g) * 0.1).to(dtype).to(D)
    index = torch.randint(-1, 3, (T,), generator=g).int().to(D)
    y = layer.adapted(x, bank, index)
    wv = R.values(layer.data, layer.scales, 384)
    frozen = layer(x.detach())
    spaced = torch.zeros(T, out + -out % 8, dtype=dtype, device=D)
    spaced[:, :out] = dy
    back = E.linear_mxfp4_input_grad(spaced[:, :out], layer.weight)
    R.check(back, *R.product(dy.cpu().double(), wv.t().contiguous(), dtype))
    want = A.adapters(frozen, x, None, bank.down, bank.up, bank.scaling, index, bank.ranks, dy, back)
    A.check(y, want["out"], "y")
    y.backward(dy)
    A.check(x.grad, want["dx"], "dx")
    A.check(bank.down.grad, want["d_down"], "d_down")
    A.check(bank.up.grad, want["d_up"], "d_up")
    # without adapters
    z = x.detach().clone().requires_grad_(True)
    layer.adapted(z).backward(dy)
    assert torch.equal(z.grad, back)
    layer.adapted(z).float().sum().backward()                     # an expanded gradient


def test_a_weight_written_before_the_backward_pass_is_refused():
    _, full = compressed(64, 64, 4, bias=False)
    layer = E.MXFP4Linear.from_ecf8(full)
    x = torch.randn(3, 64, generator=gen(1)).bfloat16().to(D).requires_grad_(True)
    y = layer.adapted(x)
    layer.data.zero_()
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_training_step_captured_while_an_eager_one_lives():
    """A captured forward and backward pass of the same leaves, replayed between eager ones."""
    _, full = compressed(96, 128, 5)
    layer = E.MXFP4Linear.from_ecf8(full)
    bank = bank_of(layer, 2, 8)
    x = torch.randn(40, 128, generator=gen(2)).bfloat16().to(D)
    dy = torch.randn(40, 96, generator=gen(3)).bfloat16().to(D)
    index = torch.randint(-1, 2, (40,), generator=gen(4)).int().to(D)
    params = [bank.down, bank.up]

    def step():
        z = x.detach().requires_grad_(True)
        y = layer.adapted(z, bank, E.AdapterPlan(index, 2))
        return [y.detach(), *torch.autograd.grad(y, [z, *params], dy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=gen(i, 5)).bfloat16())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
