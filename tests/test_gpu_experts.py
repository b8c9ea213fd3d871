"""Mixture-of-experts layers for a few tokens: routing exactly, products against float64."""
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


# ------------------------------------------------------------------ routing

def chosen(logits, top):
    """Largest first, of equal ones the lowest; NaN before everything, -inf never."""
    ids = torch.full((logits.shape[0], top), -1, dtype=torch.int32)
    for t, row in enumerate(logits.double().tolist()):
        order = sorted(range(len(row)), key=lambda e: (0, e) if row[e] != row[e] else (1, -row[e], e))
        order = [e for e in order if row[e] != -float("inf")][:top]
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
    return ids


def scores(logits, ids, score, normalise, scale):
    v = logits.double().gather(1, ids.clamp(min=0).long())
    none = ids < 0
    if score == "softmax":
        most = logits.double().amax(1, keepdim=True)
        p = torch.exp(v - most)
        total = p.masked_fill(none, 0).sum(1, keepdim=True) if normalise else torch.exp(logits.double() - most).sum(1, keepdim=True)
    else:
        p = torch.sigmoid(v)
        total = p.masked_fill(none, 0).sum(1, keepdim=True) if normalise else 1.0
    return (scale * p / total).masked_fill(none, 0)


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("T,experts,top", [(1, 1, 1), (3, 8, 2), (7, 60, 6), (64, 64, 8), (5, 65, 9), (130, 256, 8), (9, 1000, 32), (2, 1024, 1), (3, 5, 5)])
def test_route(T, experts, top, dtype):
    logits = (torch.randn(T, experts, generator=gen(T, experts)) * 3).to(dtype)
    wide = torch.full((T, experts + 3), 99.0, dtype=dtype, device=D)
    wide[:, 1:experts + 1] = logits.to(D)
    want = chosen(logits.float(), top)
    for score in ("softmax", "sigmoid"):
        for normalise, scale in ((True, 1.0), (False, 2.5)):
            for on in (logits.to(D), wide[:, 1:experts + 1]):
                ids, w = E.moe_route(on, top, score=score, normalise=normalise, scale=scale)
                assert ids.dtype == torch.int32 and torch.equal(ids.cpu(), want)
                ref = scores(logits.float(), want, score, normalise, scale)
                # exp is off by 2 ulp, twice, its argument by half an ulp of up to 30; a sum of up to 1024 terms by pairs
                assert float(((w.cpu().double() - ref).abs() - ref * 40 * 2.0 ** -23).max()) <= 1e-30


def test_route_ties_masks_and_not_a_number():
    inf, nan = float("inf"), float("nan")
    rows = [[1.0, 2.0, 2.0, 2.0, 1.0, 0.0], [0.0, -0.0, 0.0, -0.0, 0.0, 0.0], [-inf] * 6, [-inf, 3.0, -inf, -inf, 1.0, -inf],
            [-3.4e38, -inf, -3.4e38, -3.4e38, -inf, -3.4e38], [5.0, nan, 9.0, -inf, nan, 1.0]]
    logits = torch.tensor(rows)
    want = chosen(logits, 4)
    for score in ("softmax", "sigmoid"):
        ids, w = E.moe_route(logits.to(D), 4, score=score)
        assert torch.equal(ids.cpu(), want)
        w = w.cpu()
        assert bool((w[2] == 0).all()) and torch.equal(w[3] == 0, torch.tensor([False, False, True, True]))
        assert torch.equal(w[1], torch.full((4,), 0.25)) and bool(torch.isfinite(w[4]).all()) and abs(float(w[4].sum()) - 1) < 1e-6
        assert bool(torch.isnan(w[5]).any())
    ids, w = E.moe_route(torch.full((1, 6), -300.0, device=D), 2, score="sigmoid")
    assert w.tolist() == [[0.5, 0.5]]


# ------------------------------------------------------------------ products

def stacks(n, inner, K, four, seed):
    """gate, up, down as moe_few takes them, their scales, and their values in float64."""
    g = gen("stack", n, inner, K, four, seed)
    given, values, factors = [], [], []
    for rows, cols in ((inner, K), (inner, K), (K, inner)):
        if four:
            data, sc = R.random_stored((n, rows), cols, g, 117, 123)
            given.append(E.MXFP4(data.to(D), sc.to(D), cols))
            values.append(R.values(data, sc, cols))
            factors.append(None)
        else:
            b = (torch.randn(n, rows, cols, generator=g) * 40).clamp(-448, 448).to(F8)
            f = torch.rand(n, generator=g) * 2e-3 + 1e-4
            given.append(b.view(torch.uint8).to(D))
            values.append(b.double() * f.double()[:, None, None])
            factors.append(f.to(D))
    return given, dict(zip(("gate_scale", "up_scale", "down_scale"), factors)), values


CASES = [(1, 1, 1, 32, 32), (1, 4, 2, 64, 96), (1, 8, 8, 512, 160), (2, 3, 1, 96, 64), (5, 8, 2, 256, 288), (16, 4, 4, 160, 64),
         (17, 2, 2, 64, 128), (40, 2, 1, 128, 96), (64, 16, 8, 96, 128), (33, 1, 1, 288, 32), (64, 300, 8, 32, 32), (3, 1024, 6, 32, 32),
         (100, 7, 5, 64, 64), (512, 5, 1, 32, 64), (20, 64, 3, 1056, 544)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T,n,top,K,inner", CASES)
def test_layer_against_float64(T, n, top, K, inner, four, dtype):
    given, scales, values = stacks(n, inner, K, four, 1)
    g = gen(T, n, top)
    x = torch.randn(T, K, generator=g).to(dtype)
    ids, w = E.moe_route(torch.randn(T, n, generator=g).to(D), top)
    ref, tol = R.layer(x.double(), *values, ids.cpu(), w.cpu().double(), dtype)
    R.check(E.moe_few(x.to(D), *given, ids, w, **scales), ref, tol, (T, n, top, K, inner))


@pytest.mark.parametrize("K,inner", [(16, 16), (48, 80), (4112, 1040), (272, 2000)])
def test_layer_in_multiples_of_16(K, inner):
    given, scales, values = stacks(3, inner, K, False, 2)
    g = gen(K, inner)
    x = torch.randn(6, K, generator=g).to(FP)
    ids = torch.randint(0, 3, (6, 2), generator=g).int()
    w = torch.rand(6, 2, generator=g)
    ref, tol = R.layer(x.double(), *values, ids, w.double(), FP)
    R.check(E.moe_few(x.to(D), *given, ids.to(D), w.to(D), **scales), ref, tol)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T", [9, 60])
def test_layer_without_experts_twice_the_same_and_out_of_range(T, four):
    """ids of -1, past the last and large; the same expert twice for a token; a token, and then all, without any."""
    given, scales, values = stacks(4, 96, 64, four, 3)
    g = gen(T, 5)
    x = torch.randn(T, 64, generator=g).bfloat16()
    ids = torch.randint(-1, 6, (T, 3), generator=g).int()
    ids[0], ids[1], ids[2], ids[3] = torch.tensor([2, 2, 2]), torch.tensor([-1, 4, 2 ** 31 - 1]), torch.tensor([1, -2 ** 31, 1]), torch.tensor([-1] * 3)
    w = torch.randn(T, 3, generator=g)
    w[1] = float("nan")                                           # of choices that are none
    x[1, 0] = float("inf")                                        # a row that no expert takes
    ref, tol = R.layer(x.double(), *values, ids, w.double(), BF)
    wide = torch.full((T + 1, 64 + 5), 3.0, dtype=BF, device=D)
    out = wide[:T, 3:67]
    on = torch.full((T, 64 + 8), float("nan"), dtype=BF, device=D)
    on[:, 8:] = x.to(D)
    assert E.moe_few(on[:, 8:], *given, ids.to(D), w.to(D), **scales, out=out) is out
    R.check(out, ref, tol)
    assert bool((out[[1, 3]] == 0).all())
    wide[:T, 3:67] = 3.0
    assert bool((wide == 3.0).all())
    y = E.moe_few(x.to(D), *given, torch.full_like(ids, -1).to(D), w.to(D), **scales)
    assert bool((y == 0).all())


def test_layer_keeps_not_finite_rows_apart():
    given, scales, values = stacks(2, 64, 96, False, 4)
    x = torch.randn(5, 96, generator=gen(1)).bfloat16()
    x[2, 4] = float("nan")
    ids = torch.tensor([[0], [1], [0], [1], [0]], dtype=torch.int32)
    w = torch.ones(5, 1)
    ref, tol = R.layer(x.double(), *values, ids, w.double(), BF)
    R.check(E.moe_few(x.to(D), *given, ids.to(D), w.to(D), **scales), ref, tol.nan_to_num(0.0))


def test_layer_with_large_activations():
    """h past float16's and a sigmoid at both of its ends."""
    given, scales, values = stacks(2, 64, 64, False, 5)
    x = (torch.randn(4, 64, generator=gen(2)) * 1000).to(FP)
    ids = torch.tensor([[0, 1]] * 4, dtype=torch.int32)
    w = torch.full((4, 2), 2.0 ** -24)
    ref, tol = R.layer(x.double(), *values, ids, w.double(), FP)
    R.check(E.moe_few(x.to(D), *given, ids.to(D), w.to(D), **scales), ref, tol)


def test_captured_layer_replays_and_streams_agree():
    given, scales, _ = stacks(16, 256, 512, True, 6)
    x = torch.randn(12, 512, generator=gen(3)).bfloat16().to(D)
    logits = torch.randn(12, 16, generator=gen(4)).to(D)

    def step(stream=None):
        ids, w = E.moe_route(logits, 3, stream=stream)
        return E.moe_few(x, *given, ids, w, **scales, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=gen(i, 7)).bfloat16())
        logits.copy_(torch.randn(logits.shape, generator=gen(i, 8)))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [step(s) for _ in range(4) for s in sides]
    torch.cuda.synchronize()
    for y in got:
        assert torch.equal(y, want)


def test_no_tokens():
    given, scales, _ = stacks(2, 32, 32, True, 7)
    ids, w = E.moe_route(torch.empty(0, 4, device=D), 2)
    assert ids.shape == (0, 2)
    assert E.moe_few(torch.empty(0, 32, dtype=BF, device=D), *given, ids, w, **scales).shape == (0, 32)


# ------------------------------------------------------------------ the compressed layer

def test_compressed_experts_decode_route_and_run():
    n, inner, K = 5, 96, 128
    given, scales, values = stacks(n, inner, K, False, 8)
    host = [[w[e].cpu() for e in range(n)] for w in given]
    sc = torch.stack([scales[k] for k in ("gate_scale", "up_scale", "down_scale")])
    layer = E.ECF8Experts(*host, sc, device=D)
    assert layer.compressed_bytes() < 3 * n * inner * K
    for a, b in zip(layer.decode(), given):
        assert torch.equal(a, b)
    x = torch.randn(4, K, generator=gen(9)).bfloat16()
    ids, w = E.moe_route(torch.randn(4, n, generator=gen(10)).to(D), 2)
    ref, tol = R.layer(x.double(), *values, ids.cpu(), w.cpu().double(), BF)
    on = x.to(D)
    y = layer(on, ids, w)
    R.check(y, ref, tol)
    layer._pool.zero_()
    named = layer.decode(experts=ids.unique().tolist())           # only what was chosen
    assert torch.equal(layer(x.to(D), ids, w, decoded=named), y)
    four = layer.in_four_bits()
    for m, q in enumerate(four):
        stored = R.quantise((host[m][1].view(F8).float() * sc[m, 1].cpu()))
        assert torch.equal(q.data[1].cpu(), R.store(*stored)[0])
    vals = [R.values(q.data, q.scales, q.features) for q in four]
    ref, tol = R.layer(x.double(), *vals, ids.cpu(), w.cpu().double(), BF)
    R.check(E.moe_few(x.to(D), *four, ids, w), ref, tol)
    with pytest.raises(ValueError):
        layer.decode(experts=[5])
    layer.decode(experts=[0, 3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                                 # both plans are there
        again = layer(on, ids, w)
        layer.decode(experts=[3, 0])
    for _ in range(3):
        layer._pool.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, y)


def test_a_plan_is_not_made_in_a_capture(monkeypatch):
    from lossless_entropy_coded_ecf8_amd import experts as X
    given, scales, _ = stacks(2, 32, 32, False, 9)
    layer = E.ECF8Experts(*[[w[e].cpu() for e in range(2)] for w in given], torch.ones(3, 2), device=D)
    monkeypatch.setattr(X, "_capturing", lambda stream: True)
    with pytest.raises(RuntimeError):
        layer.decode()
