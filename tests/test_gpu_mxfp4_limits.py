"""Products of 4-bit weights and expert layers at the longest rows that they take."""
import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E
import mxfp4_reference as R

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)
BF, FP = torch.bfloat16, torch.float16
MOST = 1 << 20                                                    # ECF8A_MAX_FEATURES


def gen(*seed):
    return torch.Generator().manual_seed(synth.seed_of("limits", *seed))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "mx"])
@pytest.mark.parametrize("T", [1, 20, 70, 300])
def test_longest_rows_of_a_product(T, kind):
    """The values that count stand at the rows' ends and in their middle, so that float32 sums are exact."""
    g, N, K = gen(T), 37, MOST
    dtype = FP if kind == "fp16" else BF
    at = torch.tensor([0, 31, 32, 511, 512, K // 2 - 1, K // 2, K - 1025, K - 33, K - 1])
    code = torch.zeros(N, K, dtype=torch.uint8)
    code[:, at] = torch.randint(0, 16, (N, len(at)), generator=g).to(torch.uint8)
    data, scales = R.store(code, torch.full((N, K // 32), 127, dtype=torch.uint8))
    w, wv = E.MXFP4(data.to(D), scales.to(D), K), R.VALUES[code[:, at].long()]
    x = torch.zeros(T, K, dtype=dtype)
    x[:, at] = torch.randint(-4, 5, (T, len(at)), generator=g).to(dtype)
    ref = (x[:, at].double() @ wv.t()).to(dtype)
    on = E.quantize_mxfp4(x.to(D)) if kind == "mx" else x.to(D)
    assert torch.equal(E.linear_mxfp4(on, w).cpu(), ref)
    del on


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [1, 40, 130])
def test_longest_rows_of_an_input_gradient(T, dtype):
    """dy's rows as long as they may be, and dx's."""
    g = gen(T, 1)
    for N, K in ((MOST, 64), (19, MOST)):
        at = torch.tensor([0, 1, N // 2, N - 1])
        code = torch.zeros(N, K, dtype=torch.uint8)
        code[at] = torch.randint(0, 16, (4, K), generator=g).to(torch.uint8)
        data, scales = R.store(code, torch.full((N, K // 32), 127, dtype=torch.uint8))
        w = E.MXFP4(data.to(D), scales.to(D), K)
        dy = torch.zeros(T, N + -N % 8, dtype=dtype, device=D)
        some = torch.randint(-4, 5, (T, 4), generator=g).to(dtype)
        dy[:, at] = some.to(D)
        got = E.linear_mxfp4_input_grad(dy[:, :N], w).cpu()
        assert torch.equal(got, (some.float() @ R.VALUES[code[at].long()].float()).to(dtype)), (N, K)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T,K,inner", [(1, 65536, 32), (9, 65536, 64), (40, 65536, 32), (1, 32, 65536), (9, 64, 65536), (40, 32, 65536)])
def test_longest_rows_of_an_expert_layer(T, K, inner, four):
    g = gen(T, K, inner, four)
    given, values = [], []
    for rows, cols in ((inner, K), (inner, K), (K, inner)):
        if four:
            data, sc = R.random_stored((2, rows), cols, g, 117, 121)
            given.append(E.MXFP4(data.to(D), sc.to(D), cols))
            values.append(R.values(data, sc, cols))
        else:
            b = (torch.randn(2, rows, cols, generator=g) * 0.02).to(torch.float8_e4m3fn)
            given.append(b.view(torch.uint8).to(D))
            values.append(b.double())
    x = torch.randn(T, K, generator=g).bfloat16()
    ids = torch.randint(0, 2, (T, 2), generator=g).int()
    w = torch.rand(T, 2, generator=g)
    ref, tol = R.layer(x.double(), *values, ids, w.double(), BF)
    R.check(E.moe_few(x.to(D), *given, ids.to(D), w.to(D)), ref, tol, (T, K, inner))


def test_a_wide_batch_of_choices():
    """More tokens than a grid of one token a workgroup counts in 16 bits, at the ends and in between."""
    T, n = (1 << 22) + 3, 5
    g = gen(2)
    logits = torch.randn(T, n, generator=g)
    ids, w = E.moe_route(logits.to(D), 2)
    best = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(ids.cpu(), best.indices[:, :2].int())
    p = torch.exp(best.values[:, :2].double() - best.values[:, :1].double())
    ref = p / p.sum(1, keepdim=True)
    assert float((w.cpu().double() - ref).abs().max()) <= 40 * 2.0 ** -23
