"""4-bit products and expert layers in the calls that a program makes at the edges: sizes that take the largest tiles and
shares of a reduction, the limits, workspaces and results of the caller's, captured graphs side by side, refusals."""
import warnings

import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E
import lossless_entropy_coded_ecf8_amd.mxfp4 as M
import mxfp4_reference as R
from lossless_entropy_coded_ecf8_amd.binding import Ecf8Error

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)
BF, FP = torch.bfloat16, torch.float16


def gen(*seed):
    return torch.Generator().manual_seed(synth.seed_of("calls", *seed))


def weight(N, K, seed=0, lo=110, hi=128):
    data, scales = R.random_stored((N,), K, gen("w", N, K, seed), lo, hi)
    return E.MXFP4(data.to(D), scales.to(D), K), R.values(data, scales, K)


def product_is_right(kind, x, w, wv):
    dtype = FP if kind == "fp16" else BF
    x = x.to(dtype)
    if kind == "mx":
        q = E.quantize_mxfp4(x.to(D))
        R.check(E.linear_mxfp4(q, w), *R.product(R.values(q.data, q.scales, x.shape[1]), wv, BF), (kind, x.shape))
    else:
        R.check(E.linear_mxfp4(x.to(D), w), *R.product(x.double(), wv, dtype), (kind, x.shape))


@pytest.mark.parametrize("K", [32, 160, 416, 544, 672, 1056])
@pytest.mark.parametrize("T", [260, 1100])
def test_products_in_large_tiles(T, K):
    """Tiles of 256 outputs, with scales of fewer than one group, of one and of several, the last one cut."""
    w, wv = weight(6000, K)
    w2 = E.MXFP4(torch.cat([w.data, w.data, w.data[:1001]]), torch.cat([w.scales, w.scales, w.scales[:1001]]), K)
    x = torch.randn(T, K, generator=gen(T, K))
    for kind in ("bf16", "fp16", "mx"):
        product_is_right(kind, x, w, wv)
        at = x.to(FP if kind == "fp16" else BF).to(D)
        if kind == "mx":
            at = E.quantize_mxfp4(at)
        y = E.linear_mxfp4(at, w2)                                # the same rows again, in tiles of another place
        assert torch.equal(y[:, :6000], y[:, 6000:12000]) and torch.equal(y[:, 12000:], y[:, :1001])
        dtype = FP if kind == "fp16" else BF
        rows = R.values(at.data, at.scales, K) if kind == "mx" else at.cpu().double()
        R.check(y[:, 12000:], *R.product(rows, wv[:1001], dtype), (kind, T, K))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("T,N,K", [(65, 300, 96), (77, 5003, 288), (96, 14001, 1056), (97, 2000, 160), (192, 9001, 608), (285, 3000, 2080)])
def test_products_in_tiles_of_96_tokens(kind, T, N, K):
    w, wv = weight(N, K)
    product_is_right(kind, torch.randn(T, K, generator=gen(T, N, K)), w, wv)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "mx"])
@pytest.mark.parametrize("T,N,K", [(1, 1000, 8224), (4, 1000, 8224), (3, 4000, 4128), (8, 4000, 4128), (16, 130, 16416), (24, 4000, 4128),
                                   (40, 1000, 8224), (64, 3999, 4128), (70, 250, 16416), (200, 130, 6176)])
def test_products_in_shares(kind, T, N, K):
    w, wv = weight(N, K)
    product_is_right(kind, torch.randn(T, K, generator=gen(T, N)), w, wv)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "mx"])
@pytest.mark.parametrize("T,N,K", [(1100, 15361, 2080), (1100, 15361, 4128)])
def test_products_whose_last_tiles_go_in_shares(kind, T, N, K):
    """More tiles than compute units, and a few left over; some tokens of each tile, all outputs."""
    w, wv = weight(N, K)
    dtype = FP if kind == "fp16" else BF
    x = torch.randn(T, K, generator=gen(T, N)).to(dtype)
    b = torch.randn(N, generator=gen(N)).to(dtype)
    rows, given = x.double(), x.to(D)
    if kind == "mx":
        given = E.quantize_mxfp4(given)
        rows = R.values(given.data, given.scales, K)
    out = torch.full((T + 1, N + 3), 9.0, dtype=dtype, device=D)
    E.linear_mxfp4(given, w, b.to(D), out=out[:T, 2:N + 2], **({"out_dtype": dtype} if kind == "mx" else {}))
    some = list(range(0, T, 29)) + [T - 1]
    R.check(out[some][:, 2:N + 2], *R.product(rows[some], wv, dtype, b.double()), (kind, K))
    out[:T, 2:N + 2] = 9.0
    assert bool((out == 9.0).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_input_grad_whose_last_tiles_go_in_shares(dtype):
    T, N, K = 1100, 2001, 15392
    w, wv = weight(N, K)
    dy = torch.randn(T, 2008, generator=gen(T)).to(dtype)
    out = torch.full((T + 1, K + 16), 9.0, dtype=dtype, device=D)
    E.linear_mxfp4_input_grad(dy.to(D)[:, :N], w, out=out[:T, 8:K + 8])
    some = list(range(0, T, 29)) + [T - 1]
    R.check(out[some][:, 8:K + 8], *R.product(dy[some][:, :N].double(), wv.t().contiguous(), dtype), dtype)
    out[:T, 8:K + 8] = 9.0
    assert bool((out == 9.0).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,N,K", [(1100, 333, 13024), (77, 5003, 288), (97, 2000, 1056), (20, 9000, 96)])
def test_input_grad_in_large_tiles_and_shares(dtype, T, N, K):
    w, wv = weight(N, K)
    dy = torch.randn(T, -(-N // 8) * 8, generator=gen(T, N, K)).to(dtype)
    R.check(E.linear_mxfp4_input_grad(dy.to(D)[:, :N], w), *R.product(dy[:, :N].double(), wv.t().contiguous(), dtype), (T, N, K))


def test_conversion_in_several_launches():
    """More than 2^33 values, which are counted by eights and fours in 32 bits."""
    rows, K = 270000, 32768
    x = torch.zeros(rows, K, dtype=torch.uint8, device=D)
    part = torch.randint(0, 256, (4, K), generator=gen(1)).to(torch.uint8)
    part[(part & 127) == 127] = 5                                 # no NaN
    at = [0, 262143, 262144, rows - 1]
    x[at] = part.to(D)
    q = E.quantize_mxfp4(x.view(torch.float8_e4m3fn))
    want = R.store(*R.quantise(part.view(torch.float8_e4m3fn).float()))
    assert torch.equal(q.data[at].cpu(), want[0]) and torch.equal(q.scales[at].cpu(), want[1])
    del x
    for dtype in (BF, torch.float32):
        back = q.dequantize(dtype)
        assert torch.equal(back[at].cpu().double(), R.values(*want, K))
        assert not bool(back[1:262143:1000].any()) and not bool(back[262145:rows - 1:100].any())
        del back


@pytest.mark.parametrize("T", [3, 100])
def test_smallest_numbers_count(T):
    """Subnormal bfloat16 and float16 values, under weights that bring the sum back into range."""
    for dtype, unit in ((BF, 2.0 ** -133), (FP, 2.0 ** -24)):
        w, wv = weight(40, 96, 1, 227, 230) if dtype == BF else weight(40, 96, 2, 127, 130)
        x = (torch.randint(-100, 101, (T, 96), generator=gen(T)).double() * unit).to(dtype)
        assert bool((x != 0).any())
        R.check(E.linear_mxfp4(x.to(D), w), *R.product(x.double(), wv, dtype), (dtype, T))
        dy = (torch.randint(-100, 101, (T, 40), generator=gen(T, 1)).double() * unit).to(dtype)
        R.check(E.linear_mxfp4_input_grad(dy.to(D), w), *R.product(dy.double(), wv.t().contiguous(), dtype), (dtype, T))


def test_rows_as_far_apart_as_offsets_reach():
    w, wv = weight(40, 64)
    for T in (3, 66):
        for call, cols, ref in ((E.linear_mxfp4, 64, wv), (E.linear_mxfp4_input_grad, 40, wv.t().contiguous())):
            x = torch.randn(T, cols, generator=gen(T)).bfloat16()
            wide = torch.zeros(T, (1 << 22) + 8, dtype=BF, device=D)
            last = torch.as_strided(wide, (T, cols), (1 << 22, 1))
            last.copy_(x)
            R.check(call(last, w), *R.product(x.double(), ref, BF), (T, cols))
            with pytest.raises(Ecf8Error):
                call(wide[:, :cols], w)


# ------------------------------------------------------------------ experts

def stack(n, rows, cols, four, g):
    if four:
        data, sc = R.random_stored((n, rows), cols, g, 117, 123)
        return E.MXFP4(data.to(D), sc.to(D), cols), R.values(data, sc, cols)
    b = (torch.randn(n, rows, cols, generator=g) * 0.2).to(torch.float8_e4m3fn)
    return b.view(torch.uint8).to(D), b.double()


def layer(n, inner, K, four):
    g = gen("layer", n, inner, K, four)
    each = [stack(n, rows, cols, four, g) for rows, cols in ((inner, K), (inner, K), (K, inner))]
    return [w for w, _ in each], [v for _, v in each]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T,n,top,K,inner,one", [(16, 1024, 32, 32, 32, False), (512, 3, 1, 64, 32, True), (16, 40, 32, 96, 64, False),
                                                 (170, 2, 3, 32, 160, True), (48, 64, 4, 160, 32, False), (90, 64, 4, 96, 96, False)])
def test_layer_at_its_limits(T, n, top, K, inner, one, four):
    """As many experts, choices and pairs as a call takes; all pairs with one expert."""
    given, values = layer(n, inner, K, four)
    g = gen(T, n, top)
    x = torch.randn(T, K, generator=g).bfloat16()
    ids = torch.full((T, top), n - 1, dtype=torch.int32) if one else torch.randint(0, n, (T, top), generator=g).int()
    w = torch.randn(T, top, generator=g)
    R.check(E.moe_few(x.to(D), *given, ids.to(D), w.to(D)), *R.layer(x.double(), *values, ids, w.double(), BF), (T, n, top))


def test_layer_refuses_more_pairs_and_other_shapes():
    given, _ = layer(3, 32, 64, True)
    x = torch.zeros(257, 64, dtype=BF, device=D)
    ids, w = torch.zeros(257, 2, dtype=torch.int32, device=D), torch.zeros(257, 2, device=D)
    for call in (lambda: E.moe_few(x, *given, ids, w), lambda: E.moe_few(x[:4], *given, ids[:4].long(), w[:4]),
                 lambda: E.moe_few(x[:4], *given, ids[:4], w[:3]), lambda: E.moe_few(x[:4, :32], *given, ids[:4], w[:4]),
                 lambda: E.moe_few(x[:4], given[0], given[1], given[0], ids[:4], w[:4]),
                 lambda: E.moe_few(x[:4], *given, ids[:4], w[:4], gate_scale=torch.ones(3, device=D))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(Ecf8Error):                                # no choice at all
        E.moe_few(x[:4], *given, ids[:4, :0].contiguous(), w[:4, :0].contiguous())


# ------------------------------------------------------------------ the caller's memory

def calls():
    """Each product with its operands and a workspace that is large enough, as (name, call(out, workspace), operand, out)."""
    w, _ = weight(64, 16384)
    x = torch.randn(40, 16384, generator=gen(1)).bfloat16().to(D)
    v, _ = weight(16384, 64, 1)
    dy = torch.randn(40, 16384, generator=gen(2)).bfloat16().to(D)
    given, _ = layer(4, 32, 64, False)
    xm = torch.randn(6, 64, generator=gen(3)).bfloat16().to(D)
    ids, wm = E.moe_route(torch.randn(6, 4, generator=gen(4)).to(D), 2)
    q = E.quantize_mxfp4(x)
    return [("linear", lambda **k: E.linear_mxfp4(x, w, **k), x, (40, 64)), ("mx", lambda **k: E.linear_mxfp4(q, w, **k), q.data, (40, 64)),
            ("grad", lambda **k: E.linear_mxfp4_input_grad(dy, v, **k), dy, (40, 64)),
            ("moe", lambda **k: E.moe_few(xm, *given, ids, wm, **k), xm, (6, 64))]


def test_workspaces_and_results_of_the_caller():
    for name, call, operand, shape in calls():
        want = call()
        ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=D)
        out = torch.full(shape, 7.0, dtype=BF, device=D)
        for _ in range(3):                                        # what a call leaves in a workspace does not matter
            assert call(out=out, workspace=ws) is out and torch.equal(out, want), name
        flat = operand.view(torch.uint8).reshape(-1)
        for bad in (dict(workspace=ws[:256]), dict(workspace=ws[4:]), dict(workspace=flat), dict(out=operand.view(BF).reshape(-1)[:out.numel()].view(shape)),
                    dict(workspace=ws, out=ws[512:512 + 2 * out.numel()].view(BF).view(shape)), dict(out=out[:1]), dict(out=out.half())):
            with pytest.raises((ValueError, Ecf8Error)):
                call(**bad)
        assert torch.equal(call(), want), name


def test_two_streams_with_a_workspace_each():
    for name, call, _, shape in calls():
        want = call()
        sides = [torch.cuda.Stream() for _ in range(2)]
        mine = [(s, torch.empty(shape, dtype=BF, device=D), torch.empty(1 << 22, dtype=torch.uint8, device=D)) for s in sides]
        torch.cuda.synchronize()
        for _ in range(6):
            for s, out, ws in mine:
                call(out=out, workspace=ws, stream=s)
        torch.cuda.synchronize()
        for _, out, _ in mine:
            assert torch.equal(out, want), name


def test_two_graphs_side_by_side():
    """Captured on their own, replayed in turn and at once on two streams, with the same calls made eagerly between."""
    pieces = calls()
    want = [call() for _, call, _, _ in pieces]
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [call() for _, call, _, _ in pieces]
        graphs.append((graph, outs))
    sides = [torch.cuda.Stream() for _ in range(2)]
    for at_once in (False, True, True):
        for _, outs in graphs:
            for y in outs:
                y.zero_()
        eager = [call() for _, call, _, _ in pieces]
        torch.cuda.synchronize()
        for (graph, _), s in zip(graphs, sides):
            with torch.cuda.stream(s):
                graph.replay()
            if not at_once:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for y, z in zip(eager, want):
            assert torch.equal(y, z)
        for _, outs in graphs:
            for (name, *_), y, z in zip(pieces, outs, want):
                assert torch.equal(y, z), name


def test_a_layer_with_four_bit_input_says_that_it_keeps_no_gradients(monkeypatch):
    monkeypatch.setattr(M, "_warned", set())
    layer4 = E.MXFP4Linear(weight(32, 64)[0], four_bit_input=True)
    x = torch.randn(3, 64, generator=gen(5)).bfloat16().to(D).requires_grad_()
    with warnings.catch_warnings(record=True) as got:
        warnings.simplefilter("always")
        layer4(x)
        layer4(x)
    assert len(got) == 1 and "adapted" in str(got[0].message)
    layer4.adapted(x).float().sum().backward()
    assert x.grad is not None and layer4.half().scales.dtype == torch.uint8


def test_modules_brought_to_another_type_keep_their_weights():
    """Module.to changes a layer's bias, but neither the stored weights nor the experts' float32 scales."""
    x = torch.randn(4, 64, generator=gen(6)).bfloat16().to(D)
    linear = torch.nn.Linear(64, 40, device=D)
    four = E.MXFP4Linear.from_linear(linear)
    y = four(x)
    assert torch.equal(four.to(BF)(x), y) and four.bias.dtype == BF
    given, _ = layer(3, 32, 64, False)
    scales = torch.rand(3, 3, generator=gen(7)) + 0.1
    experts = E.ECF8Experts(*[[w[e].cpu() for e in range(3)] for w in given], scales, device=D)
    ids, w = E.moe_route(torch.randn(4, 3, generator=gen(8)).to(D), 2)
    y = experts(x, ids, w)
    experts.to(BF)
    assert torch.equal(experts.scales.cpu(), scales) and "scales" in dict(experts.named_buffers()) and torch.equal(experts(x, ids, w), y)
