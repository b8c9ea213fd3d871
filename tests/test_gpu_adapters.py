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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,R_", [(700, 264, 136, 16), (700, 65, 130, 9), (900, 512, 1032, 32), (900, 131, 70, 20),
                                      (1100, 136, 520, 64), (1100, 77, 129, 50), (600, 72, 136, 100)])
def test_gradients_together_and_apart(T, K, N, R_, dtype):
    """dx and the factors' gradients asked for together are bit for bit what each is alone, and meet the formula."""
    d = dev()
    s = make(d, T, K, N, R_, 5, "tokens", dtype, ranks=True, seed=T + R_)
    s["index"][s["index"] == 3] = -1                            # an adapter without a token
    plan = E.AdapterPlan(s["index"], 5)
    args = (s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan)
    kw = dict(ranks=s["ranks"], dx_base=s["dx_base"])
    dx, d_down, d_up = E.adapter_grads(*args, **kw)
    alone, none, _ = E.adapter_grads(*args, want=(True, False), **kw)
    _, down, up = E.adapter_grads(*args, want=(False, True), ranks=s["ranks"])
    assert none is None
    want = reference(s, True)
    for name, a, b in (("dx", dx, alone), ("d_down", d_down, down), ("d_up", d_up, up)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), name
        R.check(a, want[name], name)


# --------------------------------------------------------------- both ways of adding

@pytest.mark.parametrize("case", [(1, 256, 128, 4, 3), (37, 2048, 1024, 16, 5), (200, 8192, 520, 33, 40),
                                  (512, 4096, 4096, 24, 512), (300, 64, 64, 64, 2), (17, 10240, 3080, 64, 17)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_few_tokens_with_and_without_a_plan(case, dtype):
    """Up to 512 tokens an index needs no plan; both ways meet the formula (their sums run in another order)."""
    d = dev()
    T, K, N, R_, L = case
    s = make(d, T, K, N, R_, L, "tokens", dtype, seed=T)
    want = reference(s)["out"]
    R.check(add(s), want, "index")
    R.check(add(s, index=E.AdapterPlan(s["index"], L)), want, "plan")
    R.check(add(s, index=s["index"].long()), want, "int64 index")


def test_index_out_of_range_and_ranks_out_of_range():
    """Any value outside [0, L) means no adapter; ranks count as the nearest of 0 and R."""
    d = dev()
    for T, L in ((90, 4), (700, 3)):
        s = make(d, T, 192, 264, 12, L, "tokens", seed=T)
        far = s["index"].clone().long()
        far[::5] = torch.tensor([2 ** 40, -2 ** 40, L, 2 ** 31, -7], device=d)[torch.arange(far[::5].numel(), device=d) % 5]
        s["index"] = torch.where((far >= 0) & (far < L), far, -1).int()
        s["ranks"] = torch.tensor([-3, 99, 5, 12][:L], dtype=torch.int32, device=d)
        want = reference(s, True)
        R.check(add(s, index=far), want["out"])
        plan = E.AdapterPlan(far, L)
        got = E.adapter_grads(s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan, ranks=s["ranks"], dx_base=s["dx_base"])
        for name, t in zip(("dx", "d_down", "d_up"), got):
            R.check(t, want[name], name)
        assert bool((got[1][0] == 0).all()) and bool((got[2][0] == 0).all())


@pytest.mark.parametrize("T", [23, 150, 1100])
def test_in_place_touches_nothing_else(T):
    """out=base adds in place: tokens without an adapter keep their bits, as do the columns beside the slice."""
    d = dev()
    s = make(d, T, 320, 256, 16, 4, "runs", pad=24, seed=T)
    s["index"][T // 2:] = -1
    s["base"][T // 2:, ::3] = float("nan")
    buf = torch.full((T, 256 + 24 + 8), 7.0, dtype=torch.bfloat16, device=d)
    buf[:, 8:264] = s["base"]
    want = add(s)                                              # a new tensor
    before = buf.clone()
    out = E.adapter_add(buf[:, 8:264], s["x"], s["down"], s["up"], s["scaling"], s["index"], out=buf[:, 8:264])
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert torch.equal(buf[:, :8], before[:, :8]) and torch.equal(buf[:, 264:], before[:, 264:])
    assert torch.equal(buf[T // 2:].view(torch.int16), before[T // 2:].view(torch.int16))
    plain = E.adapter_add(None, s["x"], s["down"], s["up"], s["scaling"], s["index"])
    assert bool((plain[T // 2:] == 0).all())
    zero = dict(s, base=torch.zeros(T, 256, dtype=torch.bfloat16, device=d))
    assert torch.equal(plain, add(zero))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,R_,K", [(40, 10, 200), (40, 40, 2048), (900, 20, 256)])
def test_what_takes_no_part_may_hold_anything(T, R_, K, dtype):
    """NaN and infinities in rank rows past ranks, in other adapters, in other tokens and beside the rows do not reach a
    result; in a token's own row they do."""
    d = dev()
    s = make(d, T, K, 136, R_, 3, "runs", dtype, pad=8, ranks=True, seed=T + R_)
    s["ranks"][:] = torch.tensor([R_ - 3, R_ - 1, 5])
    s["index"][:] = torch.arange(T, device=d) % 2               # adapter 2 has no token
    s["index"][T // 2] = -1
    clean = {k: v.clone() if torch.is_tensor(v) and k in ("down", "up") else v for k, v in s.items()}
    for a, q in enumerate(s["ranks"].tolist()):
        s["down"][a, q:] = float("nan")
        s["up"][a, q:] = float("inf")
    s["down"][2] = float("inf")
    s["up"][2] = float("nan")
    plan = E.AdapterPlan(s["index"], 3)
    grads = lambda q: E.adapter_grads(q["dy"], q["x"], q["down"], q["up"], q["scaling"], plan, ranks=q["ranks"], dx_base=q["dx_base"])  # noqa: E731
    assert torch.equal(add(s), add(clean)) and torch.equal(add(s, index=plan), add(clean, index=plan))
    for a, b in zip(grads(s), grads(clean)):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    want = add(clean, index=plan)
    s["x"][3, 7] = float("nan")
    s["x"][T // 2, :] = float("inf")                             # a token without an adapter
    got = add(s, index=plan)
    keep = torch.arange(T, device=d) != 3
    assert bool(torch.isnan(got[3]).all()) and torch.equal(got[keep], want[keep])
    assert torch.equal(add(s)[T // 2], s["base"][T // 2])


def test_infinite_float16_values_stay_infinite():
    """A float16 factor goes into its product as two bfloat16; an infinity must not become a NaN there."""
    d = dev()
    for T in (5, 600):
        x = torch.ones(T, 64, dtype=torch.float16, device=d)
        down = torch.ones(1, 2, 64, dtype=torch.float16, device=d) / 64
        up = torch.ones(1, 2, 72, dtype=torch.float16, device=d)
        up[0, 0, 5], up[0, 1, 9] = float("inf"), float("-inf")
        out = E.adapter_add(None, x, down, up, torch.ones(1, device=d), torch.zeros(T, dtype=torch.int32, device=d))
        assert bool((out[:, 5] == float("inf")).all()) and bool((out[:, 9] == float("-inf")).all())
        rest = torch.ones(72, dtype=torch.bool)
        rest[[5, 9]] = False
        assert bool((out[:, rest.to(d)] == 2).all())


def test_no_tokens():
    d = dev()
    s = make(d, 1, 64, 64, 4, 3)
    empty = {k: s[k][:0] for k in ("base", "x", "dy", "dx_base")}
    index = s["index"][:0]
    for ix in (index, E.AdapterPlan(index, 3)):
        assert E.adapter_add(empty["base"], empty["x"], s["down"], s["up"], s["scaling"], ix).shape == (0, 64)
    dx, dd, du = E.adapter_grads(empty["dy"], empty["x"], s["down"], s["up"], s["scaling"], E.AdapterPlan(index, 3))
    assert dx.shape == (0, 64) and bool((dd == 0).all()) and bool((du == 0).all())


def test_same_bits_every_time_and_on_every_stream():
    """Two streams at once, each with its own plan and memory; every sum has a fixed order."""
    d = dev()
    s = make(d, 3000, 512, 640, 24, 5, seed=3)
    t = make(d, 300, 4096, 1032, 40, 9, "tokens", seed=4)

    def both(stream=None):
        plan = E.AdapterPlan(s["index"], 5, stream=stream)
        hidden = plan.hidden(24, stream=stream)
        out = add(s, index=plan, hidden=hidden, stream=stream)
        g = E.adapter_grads(s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan, hidden=hidden, dx_base=s["dx_base"], stream=stream)
        return [out, *g, add(t, stream=stream)]

    want = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [both(st) for _ in range(4) for st in streams]
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    plan = E.AdapterPlan(s["index"], 5, stream=streams[0])          # made on one stream, used on another
    out = add(s, index=plan, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])


def test_captured_and_replayed():
    """A captured pass with the plan inside follows its inputs on every replay; two graphs have their own memory."""
    d = dev()
    for T, N in ((2000, 512), (48, 4096)):
        s = make(d, T, 384, N, 16, 4, seed=T)
        other = make(d, T, 384, N, 16, 4, "tokens", seed=T + 1)
        names = ("base", "x", "down", "up", "index", "dy", "dx_base")

        def run():
            plan = E.AdapterPlan(s["index"], 4)
            hidden = plan.hidden(16)
            out = add(s, index=plan, hidden=hidden)
            return [out, add(s), *E.adapter_grads(s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan, hidden=hidden,
                                                  dx_base=s["dx_base"])]

        first = {k: s[k].clone() for k in names}
        want = [[t.clone() for t in run()]]
        for k in names:
            s[k].copy_(other[k])
        want.append([t.clone() for t in run()])
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs = run()
            graphs.append((g, outs))
        for k in range(6):
            src = first if k % 2 == 0 else other
            for name in names:
                s[name].copy_(src[name])
            g, outs = graphs[k // 2 % 2]
            g.replay()
            eager = run()
            torch.cuda.synchronize()
            for a, b, c in zip(outs, want[k % 2], eager):
                assert torch.equal(a, b) and torch.equal(c, b)


def test_rows_far_apart():
    """Rows 2^30 elements apart: offsets past 32 bits."""
    d = dev()
    gap = 1 << 30
    s = make(d, 3, 96, 136, 8, 2, "tokens", seed=9)
    s["index"][:] = torch.tensor([1, 0, 1])
    wide_x = torch.empty(2 * gap + 96, dtype=torch.bfloat16, device=d).as_strided((3, 96), (gap, 1))
    wide_o = torch.empty(2 * gap + 136, dtype=torch.bfloat16, device=d).as_strided((3, 136), (gap, 1))
    wide_x.copy_(s["x"])
    want = add(s)
    for index in (s["index"], E.AdapterPlan(s["index"], 2)):
        out = E.adapter_add(s["base"], wide_x, s["down"], s["up"], s["scaling"], index, out=wide_o)
        assert torch.equal(out, want)
    plan = E.AdapterPlan(s["index"], 2)
    ref = E.adapter_grads(s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan)
    got = E.adapter_grads(s["dy"], wide_x, s["down"], s["up"], s["scaling"], plan)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    del wide_x, wide_o
    torch.cuda.empty_cache()


def test_many_tokens_and_many_adapters():
    """A grouping that does not fit beside the counts in LDS, and as many adapters as a bank may have."""
    d = dev()
    for T, L, kind in ((70000, 3, "runs"), (40000, 2048, "tokens"), (13000, 2048, "runs")):
        s = make(d, T, 16, 24, 4, L, kind, seed=L)
        want = reference(s, True)
        plan = E.AdapterPlan(s["index"], L)
        hidden = plan.hidden(4)
        R.check(add(s, index=plan, hidden=hidden), want["out"], "out")
        got = E.adapter_grads(s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan, hidden=hidden, dx_base=s["dx_base"])
        for name, t in zip(("dx", "d_down", "d_up"), got):
            R.check(t, want[name], name)


def test_gradients_agree_with_differences():
    """The loss sum(c * out) is linear in x, down and up, so that a step of any size gives its slope but for rounding:
    out's (2^-8 of each value, independent of the step) and the gradients' own."""
    d = dev()
    s = make(d, 64, 128, 96, 8, 2, "runs", seed=12)
    s["index"][:] = torch.arange(64, device=d) % 2
    s["base"].zero_()
    c = torch.randn(64, 96, generator=torch.Generator().manual_seed(1)).bfloat16().to(d)
    plan = E.AdapterPlan(s["index"], 2)
    dx, dd, du = E.adapter_grads(c, s["x"], s["down"], s["up"], s["scaling"], plan)
    f = lambda q: add(q, index=plan).double()  # noqa: E731
    g = torch.Generator().manual_seed(2)
    for name, grad in (("x", dx), ("down", dd), ("up", du)):
        step = torch.randn(s[name].shape, generator=g).to(s[name].dtype).to(d)
        up_, down_ = dict(s, **{name: step}), dict(s, **{name: -step})    # linear: the value at a step is the slope
        hi, lo = f(up_), f(down_)
        slope = float((c.double() * (hi - lo)).sum() / 2)
        terms = grad.double() * step.double()
        # each out value is off by 2^-8 of itself, each gradient value by 2^-8 of itself, and 2^-12 for the float32 sums
        bound = float((c.double().abs() * (hi.abs() + lo.abs()) / 2).sum() * (2 ** -8 + 2 ** -12) + terms.abs().sum() * (2 ** -8 + 2 ** -12))
        assert abs(slope - float(terms.sum())) <= bound, name


def test_refusals():
    d = dev()
    s = make(d, 12, 64, 72, 4, 3)
    ok = dict(base=s["base"], x=s["x"], down=s["down"], up=s["up"], scaling=s["scaling"], index=s["index"])
    call = lambda **k: E.adapter_add(**{**ok, **k})  # noqa: E731
    call()
    for bad in (dict(x=s["x"].float()), dict(x=s["x"][:, :60]), dict(x=s["x"].cpu()), dict(base=s["base"].half()),
                dict(base=s["base"].t().contiguous().t()), dict(up=s["up"].half()), dict(up=s["up"][:2]),
                dict(down=s["down"].transpose(1, 2)), dict(scaling=s["scaling"].double()), dict(scaling=s["scaling"][:2]),
                dict(index=s["index"].float()), dict(index=s["index"].cpu()), dict(index=s["index"][:11]),
                dict(index=s["index"][::2]), dict(ranks=torch.ones(3, dtype=torch.int64, device=d)),
                dict(x_scale=torch.tensor(1.0, device=d)), dict(out=s["base"][:, :71]),
                dict(out=torch.empty(12, 72, dtype=torch.bfloat16, device=d).expand(12, 72)[:11]),
                dict(index=E.AdapterPlan(s["index"], 4)), dict(hidden=torch.empty(1 << 20, dtype=torch.uint8, device=d))):
        with pytest.raises((ValueError, E.Ecf8Error)):
            call(**bad)
    rows = torch.zeros(13, 72, dtype=torch.bfloat16, device=d)
    with pytest.raises(ValueError):                               # out one row further on than base
        call(base=rows[:12], out=rows[1:])
    square = torch.zeros(12, 64, dtype=torch.bfloat16, device=d)
    up = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=d)
    with pytest.raises(ValueError):                               # out over x
        call(base=None, x=square, up=up, out=square)
    both = torch.zeros(12, 128, dtype=torch.bfloat16, device=d)    # out beside x in one buffer: apart
    E.adapter_add(None, both[:, :64], s["down"], up, s["scaling"], s["index"], out=both[:, 64:])
    plan = E.AdapterPlan(s["index"], 3)
    with pytest.raises(ValueError):
        E.adapter_add(**{**ok, "index": plan}, hidden=torch.empty(16, dtype=torch.uint8, device=d))
    with pytest.raises(ValueError):
        E.adapter_grads(s["dy"], None, s["down"], s["up"], s["scaling"], plan)
    with pytest.raises(ValueError):
        E.adapter_grads(s["dy"].float(), s["x"], s["down"], s["up"], s["scaling"], plan)
    with pytest.raises(E.Ecf8Error):
        E.AdapterPlan(s["index"], 0)
    with pytest.raises(E.Ecf8Error):
        E.AdapterPlan(s["index"], 2049)
    only = E.adapter_grads(s["dy"], None, s["down"], s["up"], s["scaling"], plan, want=(True, False))
    assert only[1] is None and only[2] is None and only[0].shape == (12, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_infinite_rows_give_infinite_gradients(dtype):
    """An infinity in a token's own row reaches its adapter's gradient as an infinity in that column, and nothing else
    becomes a NaN where the formula has none (h and z are positive here)."""
    d = dev()
    for T in (20, 700):
        x, down = torch.ones(T, 80, dtype=dtype, device=d), torch.full((2, 3, 80), 0.125, dtype=dtype, device=d)
        dy, up = torch.ones(T, 88, dtype=dtype, device=d), torch.full((2, 3, 88), 0.25, dtype=dtype, device=d)
        index = (torch.arange(T, device=d) % 2).int()
        plan = E.AdapterPlan(index, 2)
        one = torch.ones(2, device=d)
        hidden = plan.hidden(3)
        E.adapter_add(None, x, down, up, one, plan, hidden=hidden)
        x[4, 7] = float("inf")                                   # token 4: adapter 0
        _, dd, du = E.adapter_grads(dy, x, down, up, one, plan, hidden=hidden)
        assert bool((dd[0, :, 7] == float("inf")).all())
        rest = torch.arange(80, device=d) != 7
        assert bool(torch.isfinite(dd[0][:, rest]).all()) and bool(torch.isfinite(dd[1]).all()) and bool(torch.isfinite(du).all())
