"""Adapters on compressed layers as they are used: serving through ECF8Linear and DecodePipeline, training through
ECF8Linear.adapted, gradients clipped together."""
import math

import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import pipeline as P
import adapter_reference as R

pytestmark = pytest.mark.gpu


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def layer_of(d, out, inn, seed, bias=False):
    w = torch.from_numpy(synth.small_stable(out * inn, 1.8, seed)).view(out, inn)
    b = torch.randn(out, generator=torch.Generator().manual_seed(seed)).bfloat16() if bias else None
    return w.to(d), E.ECF8Linear(w, scale=2e-4, bias=b, device=d)


def bank_of(layer, n, rank, seed, ranks=None, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    bank = E.AdapterBank(n, rank, layer.in_features, layer.out_features, scaling=torch.linspace(0.5, 1.5, n), ranks=ranks,
                         dtype=dtype, device=layer.device)
    with torch.no_grad():
        bank.down.copy_((torch.randn(bank.down.shape, generator=g) / layer.in_features ** 0.5).to(dtype))
        bank.up.copy_((torch.randn(bank.up.shape, generator=g) * 0.1).to(dtype))
    return bank


def inputs(d, T, K, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, K, generator=g) * 4).clamp(-448, 448).to(torch.float8_e4m3fn).to(d), torch.tensor(0.25, device=d)


@pytest.mark.parametrize("T", [1, 48, 700])
def test_serving_layer_adds_its_adapters(T):
    d = dev()
    w, layer = layer_of(d, 320, 512, 1, bias=True)
    bank = bank_of(layer, 4, 12, 2, ranks=[12, 3, 0, 7])
    x, s = inputs(d, T, 512, T)
    index = torch.randint(-1, 4, (T,), generator=torch.Generator().manual_seed(T)).int().to(d)
    base = P.linear_fp8(x, s, w, layer.w_scale, layer.bias)
    assert torch.equal(layer(x, s), base)                          # without adapters: as before
    want = R.adapters(base, x, s, bank.down, bank.up, bank.scaling, index, bank.ranks)["out"]
    for ix in (index, E.AdapterPlan(index, 4)):
        got = layer(x, s, adapters=bank, index=ix)
        R.check(got, want)
        assert torch.equal(got[index < 0], base[index < 0])
    with pytest.raises(ValueError):
        layer(x, s, adapters=bank)


@pytest.mark.parametrize("T,slots,ahead", [(37, 3, 2), (37, 1, 0), (900, 2, 1)])
def test_pipeline_with_adapters_matches_its_layers(T, slots, ahead):
    d = dev()
    shapes = [(512, 512), (128, 512), (1024, 512), (512, 1024), (512, 512)]
    ws, layers = zip(*[layer_of(d, o, k, i) for i, (o, k) in enumerate(shapes)])
    banks = [None if i == 2 else bank_of(l, 3, 8, i) for i, l in enumerate(layers)]
    ins = [inputs(d, T, l.in_features, 10 + i) for i, l in enumerate(layers)]
    xs, ss = [i[0] for i in ins], [i[1] for i in ins]
    index = torch.randint(-1, 3, (T,), generator=torch.Generator().manual_seed(5)).int().to(d)
    pipe = E.DecodePipeline(layers, slots=slots, ahead=ahead)
    plain = pipe.run(xs, ss)
    for i, o in enumerate(plain):
        assert torch.equal(o, P.linear_fp8(xs[i], ss[i], ws[i], layers[i].w_scale))
    for _ in range(2):
        outs = pipe.run(xs, ss, adapters=banks, index=index)
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            base = P.linear_fp8(xs[i], ss[i], ws[i], layers[i].w_scale)
            if banks[i] is None:
                assert torch.equal(o, base)
            else:
                R.check(o, R.adapters(base, xs[i], ss[i], banks[i].down, banks[i].up, banks[i].scaling, index, None)["out"], i)
    with pytest.raises(ValueError):
        pipe.run(xs, ss, adapters=banks[:2], index=index)
    with pytest.raises(ValueError):
        pipe.run(xs, ss, adapters=banks)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [5, 130, 800])
def test_training_layer_against_formula(T, dtype):
    """y, dx, d_down and d_up of one layer for a given dy: the frozen weight's part of dx is rounded once, then the
    adapters' part is added and rounded again."""
    d = dev()
    w, layer = layer_of(d, 272, 384, 3, bias=True)
    bank = bank_of(layer, 3, 10, 4, ranks=[10, 4, 9], dtype=dtype)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 384, generator=g).to(dtype).to(d).requires_grad_(True)
    dy = (torch.randn(T, 272, generator=g) * 0.1).to(dtype).to(d)
    index = torch.randint(-1, 3, (T,), generator=g).int().to(d)
    y = layer.adapted(x, bank, index)
    xq, s = E.quantize_e4m3(x)
    base = P.linear_fp8(xq, s, w, layer.w_scale, layer.bias, out_dtype=dtype)
    frozen = E.linear_fp8_input_grad(dy, w, layer.w_scale)
    want = R.adapters(base, x, None, bank.down, bank.up, bank.scaling, index, bank.ranks, dy, frozen)
    R.check(y, want["out"], "y")
    y.backward(dy)
    R.check(x.grad, want["dx"], "dx")
    R.check(bank.down.grad, want["d_down"], "d_down")
    R.check(bank.up.grad, want["d_up"], "d_up")
    assert bank.scaling.grad is None and layer.bias.grad is None
    # a kept weight gives the same bits, and x alone or the adapters alone can be asked for
    x2 = x.detach().clone().requires_grad_(True)
    (a,) = torch.autograd.grad(layer.adapted(x2, bank, E.AdapterPlan(index, 3), weight_u8=w), [x2], dy)
    assert torch.equal(a, x.grad)
    b, c = torch.autograd.grad(layer.adapted(x.detach(), bank, index), [bank.down, bank.up], dy)
    assert torch.equal(b, bank.down.grad) and torch.equal(c, bank.up.grad)


def test_expanded_gradients_and_changed_parameters():
    """The gradient of a sum is one value, expanded; a parameter changed between forward and backward is refused."""
    d = dev()
    w, layer = layer_of(d, 64, 128, 6)
    bank = bank_of(layer, 1, 4, 7)
    x = torch.randn(9, 128, device=d).bfloat16().requires_grad_(True)
    index = torch.zeros(9, dtype=torch.int64, device=d)
    layer.adapted(x, bank, index).sum().backward()
    first = x.grad.clone()
    x.grad = None
    layer.adapted(x, bank, index).backward(torch.ones(9, 64, dtype=torch.bfloat16, device=d))
    assert torch.equal(x.grad, first)
    y = layer.adapted(x, bank, index)
    with torch.no_grad():
        bank.up.add_(1)
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_a_training_step_of_stacked_layers():
    """Two compressed layers, adapters on both, one loss: gradients flow through the upper one's frozen weight, all are
    clipped together, and a step against the gradient lowers the loss as its slope says (to first order)."""
    d = dev()
    _, lower = layer_of(d, 256, 128, 8)
    _, upper = layer_of(d, 64, 256, 9)
    banks = [bank_of(lower, 2, 8, 10), bank_of(upper, 2, 8, 11)]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(96, 128, generator=g).bfloat16().to(d)
    target = torch.randn(96, 64, generator=g).to(d)
    index = (torch.arange(96, device=d) // 48).int()
    plan = E.AdapterPlan(index, 2)
    y = upper.adapted(lower.adapted(x, banks[0], plan), banks[1], plan)
    loss = ((y.float() - target) ** 2).mean()
    loss.backward()
    params = [p for b in banks for p in (b.down, b.up)]
    before = [p.grad.clone() for p in params]
    # the chain by hand: the upper layer's gradient of its input is the lower one's dy
    dy = (2 * (y.detach().float() - target) / y.numel()).bfloat16()
    h = lower.adapted(x, banks[0], plan).detach()
    dx, dd, du = E.adapter_grads(dy, h, banks[1].down.detach(), banks[1].up.detach(), banks[1].scaling, plan,
                                 dx_base=E.linear_fp8_input_grad(dy, upper.decoded_weight(), upper.w_scale))
    assert torch.equal(dd, before[2]) and torch.equal(du, before[3])
    _, dd, du = E.adapter_grads(dx, x, banks[0].down.detach(), banks[0].up.detach(), banks[0].scaling, plan, want=(False, True))
    assert torch.equal(dd, before[0]) and torch.equal(du, before[1])
    want = math.sqrt(sum(float((b.double() ** 2).sum()) for b in before))
    norm = E.clip_adapter_grads(banks, want / 2)
    assert abs(float(norm) / want - 1) <= 2.0 ** -23
    for p, b in zip(params, before):
        # half of a value is exact but for the 1e-6 in the factor and its rounding to float32
        assert bool(((p.grad.double() - b.double() / 2).abs() <= b.double().abs() * (2.0 ** -8 + 1e-6 / want + 2.0 ** -23)).all())


def test_serving_step_captured():
    """A decode step of a layer with adapters in a graph: other inputs and another index on each replay."""
    d = dev()
    w, layer = layer_of(d, 512, 1024, 12)
    bank = bank_of(layer, 6, 16, 13)
    x, s = inputs(d, 16, 1024, 1)
    index = torch.zeros(16, dtype=torch.int32, device=d)
    layer(x, s, adapters=bank, index=index)                        # the weight's buffer, once
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(x, s, adapters=bank, index=index)
    for k in range(4):
        x.copy_(inputs(d, 16, 1024, 20 + k)[0])
        index.copy_(torch.randint(-1, 6, (16,), generator=torch.Generator().manual_seed(k)).int())
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, layer(x, s, adapters=bank, index=index))
        torch.cuda.synchronize()
