"""Low-rank adapters of many requests beside a shared projection, against the formulas in 64 bits."""
import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
import adapter_reference as R

pytestmark = pytest.mark.gpu


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def index_of(kind, T, L, g):
    if kind == "one":
        return torch.full((T,), L - 1)
    if kind == "none":
        return torch.full((T,), -1)
    if kind == "tokens":
        return torch.randint(-1, L, (T,), generator=g)
    got = []
    while len(got) < T:                                        # runs of one adapter, some without
        got += [int(torch.randint(-1, L, (1,), generator=g))] * int(torch.randint(1, max(2, T // 3 + 2), (1,), generator=g))
    return torch.tensor(got[:T])


def wide(t, pad, d):
    if not pad:
        return t.to(d)
    w = torch.full((t.shape[0], t.shape[1] + pad), float("nan")).to(t.dtype).to(d)
    w[:, :t.shape[1]] = t.to(d)
    return w[:, :t.shape[1]]


def make(d, T, K, N, R_, L, kind="runs", dtype=torch.bfloat16, e4m3=False, pad=0, ranks=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = dict(base=wide(rnd(T, N).to(dtype), pad, d), down=(rnd(L, R_, K) / K ** 0.5).to(dtype).to(d),
             up=(rnd(L, R_, N) * 0.3).to(dtype).to(d), scaling=(torch.rand(L, generator=g) * 3 - 1).to(d),
             index=index_of(kind, T, L, g).to(torch.int32).to(d),
             ranks=torch.randint(0, R_ + 1, (L,), generator=g, dtype=torch.int32).to(d) if ranks else None, x_scale=None,
             dy=wide((rnd(T, N) * 0.1).to(dtype), pad, d), dx_base=wide(rnd(T, K).to(dtype), pad, d))
    x = rnd(T, K)
    if e4m3:
        s["x_scale"] = torch.tensor(0.37, device=d)
        s["x"] = wide(x.to(torch.float8_e4m3fn), pad, d)
    else:
        s["x"] = wide(x.to(dtype), pad, d)
    return s


def add(s, **kw):
    kw = {"index": s["index"], **kw}
    return E.adapter_add(s["base"], s["x"], s["down"], s["up"], s["scaling"], ranks=s["ranks"], x_scale=s["x_scale"], **kw)


def reference(s, grads=False):
    return R.adapters(s["base"], s["x"], s["x_scale"], s["down"], s["up"], s["scaling"], s["index"], s["ranks"],
                      s["dy"] if grads else None, s["dx_base"] if grads else None)


CASES = [  # T, K, N, R, L, index, pad, ranks
    (1, 64, 64, 1, 1, "one", 0, False),
    (1, 4096, 1024, 16, 8, "one", 0, False),
    (2, 7, 3, 2, 2, "tokens", 0, False),
    (3, 1, 1, 1, 1, "one", 0, False),
    (15, 136, 128, 16, 3, "runs", 8, False),
    (16, 192, 520, 17, 2, "runs", 0, True),
    (17, 200, 127, 8, 1, "one", 0, False),
    (33, 264, 1000, 24, 4, "runs", 5, True),
    (40, 128, 640, 32, 1, "one", 0, False),
    (48, 320, 136, 33, 2, "one", 16, False),
    (63, 64, 512, 48, 3, "tokens", 0, True),
    (64, 2048, 513, 64, 64, "tokens", 0, False),
    (65, 72, 264, 65, 2, "runs", 0, True),
    (130, 96, 1544, 100, 5, "runs", 0, False),
    (77, 333, 129, 256, 2, "runs", 0, True),
    (257, 512, 384, 16, 300, "tokens", 0, False),
    (700, 1024, 256, 16, 7, "runs", 0, True),
    (1500, 256, 1088, 40, 3, "runs", 8, False),
    (200, 128, 128, 8, 5, "none", 0, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_add_against_formula(case, dtype):
    d = dev()
    T, K, N, R_, L, kind, pad, ranks = case
    for e4m3 in (False, True):
        s = make(d, T, K, N, R_, L, kind, dtype, e4m3, pad, ranks, seed=T + R_)
        out = add(s)
        R.check(out, reference(s)["out"], (case, e4m3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES + [(2500, 96, 160, 16, 2, "runs", 0, False), (5000, 64, 72, 8, 3, "runs", 0, True)],
                         ids=str)
def test_grads_against_formula(case, dtype):
    d = dev()
    T, K, N, R_, L, kind, pad, ranks = case
    s = make(d, T, K, N, R_, L, kind, dtype, False, pad, ranks, seed=T + R_ + 1)
    plan = E.AdapterPlan(s["index"], L)
    hidden = plan.hidden(R_)
    out = add(s, index=plan, hidden=hidden)
    want = reference(s, True)
    R.check(out, want["out"], "out")
    args = (s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan)
    got = E.adapter_grads(*args, hidden=hidden, ranks=s["ranks"], dx_base=s["dx_base"])
    for name, t in zip(("dx", "d_down", "d_up"), got):
        R.check(t, want[name], name)
    again = E.adapter_grads(*args, ranks=s["ranks"], dx_base=s["dx_base"])     # h computed again from x
    for a, b in zip(got, again):
        assert torch.equal(a, b)
