"""The measured cases of the operators beside a compressed layer.

`ECF8Linear` keeps a frozen FP8 E4M3 weight.  What a user serves and trains next to it:

  add         low-rank adapters of many requests added to the shared projection's output
  train       the same for a training pass: the addition, then the gradients of the projection's
              input and of both adapter factors
  input_grad  the gradient that a frozen E4M3 weight passes back to its input
  clip        the global norm of many gradients, and the gradients scaled to a largest norm

`run` computes each in elementary torch operations, or, where `own` is set, through the package.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one request through a 4096-wide projection: latency alone
        dict(name="add_one_token", op="add", tokens=1, k=4096, n=4096, rank=16, adapters=8, dtype="bf16", x="bf16",
             index="tokens", bare=0.0, mixed_ranks=False, pad=0),
        # a decode step of 64 requests, most with an adapter of their own, at the 8192-wide output projection
        dict(name="add_decode_64", op="add", tokens=64, k=8192, n=8192, rank=16, adapters=64, dtype="bf16", x="bf16",
             index="tokens", bare=0.1, mixed_ranks=False, pad=0),
        # decode steps and short prompts in one batch, activations already in E4M3, a key projection that
        # writes its columns of a fused buffer, adapters of several ranks in one bank
        dict(name="add_mixed_e4m3", op="add", tokens=331, k=4096, n=1024, rank=24, adapters=9, dtype="fp16", x="e4m3",
             index="mixed", bare=0.2, mixed_ranks=True, pad=512),
        # prompts of several requests through the 4096 to 14336 projection
        dict(name="add_prompts", op="add", tokens=8192, k=4096, n=14336, rank=32, adapters=8, dtype="bf16", x="bf16",
             index="prompts", bare=0.1, mixed_ranks=False, pad=0),
        # one short odd sequence in training, sizes off every tile
        dict(name="train_ragged", op="train", tokens=77, k=1000, n=1364, rank=6, adapters=3, dtype="fp16", x="fp16",
             index="prompts", bare=0.0, mixed_ranks=True, pad=0),
        # a training batch with several adapters at a 4096-wide projection
        dict(name="train_4096", op="train", tokens=4096, k=4096, n=4096, rank=16, adapters=4, dtype="bf16", x="bf16",
             index="prompts", bare=0.0, mixed_ranks=False, pad=0),
        # one adapter of high rank at the diffusion block's widest projection, a long batch
        dict(name="train_long_rank64", op="train", tokens=16384, k=5120, n=13824, rank=64, adapters=1, dtype="bf16",
             x="bf16", index="one", bare=0.0, mixed_ranks=False, pad=0),
        # a few tokens: the weight alone has to be read
        dict(name="input_grad_24", op="input_grad", tokens=24, k=4096, n=14336, dtype="bf16"),
        # an ordinary batch of odd length in fp16
        dict(name="input_grad_1001", op="input_grad", tokens=1001, k=4096, n=4096, dtype="fp16"),
        # a full batch at the 8192 to 28672 projection
        dict(name="input_grad_4096", op="input_grad", tokens=4096, k=8192, n=28672, dtype="bf16"),
        # the adapters of one block: 14 gradients
        dict(name="clip_block", op="clip", tensors=14, smallest=16384, largest=458752, dtype="bf16", max_norm=0.5),
        # the adapters of 40 blocks
        dict(name="clip_model", op="clip", tensors=560, smallest=16384, largest=458752, dtype="bf16", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.3 else max(8, w // 8 * 8)


def draw(rng):
    op = rng.choice(["add", "add", "train", "train", "input_grad", "clip"])
    if op == "input_grad":
        k, n = (16 * _log(rng, 1, 896) for _ in range(2))
        most = 4096 * 8192 * 28672 // 4
        return dict(op=op, tokens=_log(rng, 1, max(1, min(8192, most // (k * n)))), k=k, n=n,
                    dtype=rng.choice(["bf16", "fp16"]))
    if op == "clip":
        small = _log(rng, 1, 16384)
        return dict(op=op, tensors=_log(rng, 1, 560), smallest=small, largest=small + _log(rng, 1, 400000),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), max_norm=rng.choice([0.1, 1.0, 1e6]))
    dtype = rng.choice(["bf16", "fp16"])
    return dict(op=op, tokens=_log(rng, 1, 8192), k=_width(rng, 48, 8192), n=_width(rng, 48, 8192),
                rank=_log(rng, 1, 64), adapters=_log(rng, 1, 16), dtype=dtype,
                x=rng.choice([dtype, "e4m3"]) if op == "add" else dtype,
                index=rng.choice(["tokens", "mixed", "prompts", "one"]), bare=rng.choice([0.0, 0.0, 0.1, 0.5]),
                mixed_ranks=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 512, 5]))


# ------------------------------------------------------------------ inputs

def _index(case, seed):
    """The adapter of each token (-1: none): single tokens, prompts of one request each, or both."""
    rng, t, kind = random.Random(seed), case["tokens"], case["index"]
    pick = lambda: -1 if rng.random() < case["bare"] else rng.randrange(case["adapters"])  # noqa: E731
    if kind == "one":
        a = rng.randrange(case["adapters"])
        return [a] * t
    got = [pick() for _ in range(t if kind == "tokens" else t // 4 if kind == "mixed" else 0)]
    while len(got) < t:
        got += [pick()] * rng.randint(1, max(1, t // 6))
    return got[:t]


def _sizes(case):
    """Elements of each gradient: spread over [smallest, largest], whole 16-byte units but for every ninth."""
    m, lo, hi = case["tensors"], case["smallest"], case["largest"]
    at = [lo * (hi / lo) ** ((i * 37 % m) / max(1, m - 1)) for i in range(m)]
    return [max(1, int(s) // 8 * 8) if i % 9 else max(1, int(s) + 3) for i, s in enumerate(at)]


def _padded(t, pad, rnd):
    """`t` as the leading columns of a wider buffer."""
    if not pad:
        return t
    wide = rnd(t.shape[0], t.shape[1] + pad).to(t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    dt, s = TYPES[case["dtype"]], dict(case)
    if case["op"] == "clip":
        sizes = _sizes(case)
        s["grads"] = [(rnd(m) * 10 ** random.Random(seed * 1000 + i).uniform(-4, -2)).to(dt) for i, m in enumerate(sizes)]
        unit = 16 // s["grads"][0].element_size()
        s["gaps"] = [torch.zeros(-m % unit, dtype=dt, device="cuda") for m in sizes]
        # the clipped gradients go into one bucket, each from a 16-byte border on
        s["bucket"] = torch.zeros(sum(m + -m % unit for m in sizes), dtype=dt, device="cuda")
        at, s["out"] = 0, []
        for m in sizes:
            s["out"].append(s["bucket"][at:at + m])
            at += m + -m % unit
        if own:
            import lossless_entropy_coded_ecf8_amd as E
            s["plan"] = E.GradClip(s["grads"], out=s["out"])     # the gradients' addresses, as kept from step to step
        return s
    t, k, n = case["tokens"], case["k"], case["n"]
    if case["op"] == "input_grad":
        s["dy"] = (rnd(t, n) * 1e-2).to(dt)
        w = rnd(n, k)
        w = w * (1 + w.square())                                  # heavy tails, as trained weights have
        s["w"] = (w * (448 / w.abs().max())).to(torch.float8_e4m3fn).view(torch.uint8)
        s["w_scale"] = torch.tensor(0.02 / 448 * 8, device="cuda")
        return s
    a, r = case["adapters"], case["rank"]
    s["index"] = torch.tensor(_index(case, seed), dtype=torch.int32, device="cuda")
    s["down"] = (rnd(a, r, k) / math.sqrt(k)).to(dt)
    s["up"] = (rnd(a, r, n) * 0.05).to(dt)
    s["scaling"] = torch.rand(a, generator=g, device="cuda") * 2 + 0.25
    s["ranks"] = None
    if case["mixed_ranks"]:
        s["ranks"] = torch.randint(1, r + 1, (a,), generator=g, device="cuda", dtype=torch.int32)
    x = rnd(t, k)
    s["x_scale"] = None
    if case["x"] == "e4m3":
        s["x_scale"] = (x.abs().max() / 448).reshape(())
        x = x / s["x_scale"]
    s["x"] = _padded(x.to(TYPES[case["x"]]), case["pad"], rnd)
    s["base"] = _padded(rnd(t, n).to(dt), case["pad"], rnd)
    if case["op"] == "train":
        s["dy"] = (rnd(t, n) * 1e-2).to(dt)
        s["dx_base"] = (rnd(t, k) * 1e-2).to(dt)
    return s


# ------------------------------------------------------------------ one pass

def _pick(s):
    """(T, adapters * rank): whether a token's adapter has this row."""
    a, r, _ = s["down"].shape
    dev = s["down"].device
    mine = s["index"][:, None] == torch.arange(a, device=dev)
    has = torch.ones(a, r, dtype=torch.bool, device=dev)
    if s["ranks"] is not None:
        has = torch.arange(r, device=dev) < s["ranks"][:, None]
    return (mine[:, :, None] & has).reshape(-1, a * r)


def _low(v, rows, s, pick):
    """The scaled product of each token with its adapter's rows, zero elsewhere: all adapters in one product."""
    a, r, c = rows.shape
    z = v @ rows.reshape(a * r, c).float().t() * s["scaling"].repeat_interleave(r)
    return torch.where(pick, z, torch.zeros((), device=z.device))


def _plain_add(s, pick):
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"]
    h = _low(x, s["down"], s, pick)
    a, r, n = s["up"].shape
    return x, h, (s["base"].float() + h @ s["up"].reshape(a * r, n).float()).to(s["base"].dtype)


def run(s):
    if own:
        import lossless_entropy_coded_ecf8_amd as E
        if s["op"] == "clip":
            norm = s["plan"].run(s["max_norm"])
            return [s["bucket"], norm]
        if s["op"] == "input_grad":
            return E.linear_fp8_input_grad(s["dy"], s["w"], s["w_scale"])
        if s["op"] == "add":
            return E.adapter_add(s["base"], s["x"], s["down"], s["up"], s["scaling"], s["index"], ranks=s["ranks"],
                                 x_scale=s["x_scale"])
        plan = E.AdapterPlan(s["index"], s["adapters"])
        hidden = plan.hidden(s["rank"])
        out = E.adapter_add(s["base"], s["x"], s["down"], s["up"], s["scaling"], plan, ranks=s["ranks"], hidden=hidden)
        dx, d_down, d_up = E.adapter_grads(s["dy"], s["x"], s["down"], s["up"], s["scaling"], plan, hidden=hidden,
                                           ranks=s["ranks"], dx_base=s["dx_base"])
        return [out, dx, d_down, d_up]
    if s["op"] == "clip":
        flat = torch.cat([p for g, z in zip(s["grads"], s["gaps"]) for p in (g, z)])
        norm = flat.double().square().sum().sqrt()
        scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        return [(flat.float() * scale).to(flat.dtype), norm.float()]
    if s["op"] == "input_grad":
        w = s["w"].view(torch.float8_e4m3fn).float()
        return ((s["dy"].float() @ w) * s["w_scale"]).to(s["dy"].dtype)
    pick = _pick(s)
    x, h, out = _plain_add(s, pick)
    if s["op"] == "add":
        return out
    dt, (a, r, k), n = s["base"].dtype, s["down"].shape, s["up"].shape[2]
    dy = s["dy"].float()
    z = _low(dy, s["up"], s, pick)
    dx = (s["dx_base"].float() + z @ s["down"].reshape(a * r, k).float()).to(dt)
    return [out, dx, (z.t() @ x).to(dt).reshape(a, r, k), (h.t() @ dy).to(dt).reshape(a, r, n)]


# ------------------------------------------------------------------ what it cannot do without

def work(case):
    if case["op"] == "clip":
        m, size = sum(_sizes(case)), {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": 2 * m * size + 4, "flops": 3 * m}
    t, k, n = case["tokens"], case["k"], case["n"]
    if case["op"] == "input_grad":
        return {"bytes": 2 * t * n + n * k + 2 * t * k, "flops": 2 * t * n * k}
    r = case["rank"]
    used = 1 if case["index"] == "one" else min(case["adapters"], t)
    factors = 2 * used * r * (k + n)
    add = (1 if case["x"] == "e4m3" else 2) * t * k + 4 * t * n + 4 * t
    if case["op"] == "add":
        return {"bytes": add + factors, "flops": 2 * t * r * (k + n)}
    return {"bytes": add + 2 * t * n + 4 * t * k + factors + 2 * case["adapters"] * r * (k + n),
            "flops": 6 * t * r * (k + n)}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3_values(device):
    """The value of each E4M3 byte, from its bits: sign, 4 exponent bits of bias 7, 3 mantissa bits, no infinities."""
    got = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        got.append(math.nan if b & 127 == 127 else -v if b & 128 else v)
    return torch.tensor(got, dtype=torch.float64, device=device)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = math.fsum(float((g.double() ** 2).sum()) for g in s["grads"])
        norm = math.sqrt(total)
        scale = min(1.0, case["max_norm"] / (norm + 1e-6))
        bucket = torch.zeros(s["bucket"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for g, z in zip(s["grads"], s["gaps"]):
            bucket[at:at + g.numel()] = g.double() * scale
            at += g.numel() + z.numel()
        return [bucket, norm]
    if case["op"] == "input_grad":
        w = _e4m3_values("cuda")[s["w"].long()]
        return torch.mm(s["dy"].double(), w) * float(s["w_scale"])
    x = s["x"].double() if s["x_scale"] is None else _e4m3_values("cuda")[s["x"].view(torch.uint8).long()] * float(s["x_scale"])
    out = s["base"].double()
    train = case["op"] == "train"
    if train:
        dy, dx = s["dy"].double(), s["dx_base"].double()
        d_down, d_up = (torch.zeros(s[w].shape, dtype=torch.float64, device="cuda") for w in ("down", "up"))
    for a in range(case["adapters"]):
        rows = (s["index"] == a).nonzero()[:, 0]
        q = case["rank"] if s["ranks"] is None else int(s["ranks"][a])
        down, up, c = s["down"][a, :q].double(), s["up"][a, :q].double(), float(s["scaling"][a])
        h = torch.mm(x[rows], down.t().contiguous()) * c
        out[rows] += torch.mm(h, up)
        if train:
            z = torch.mm(dy[rows], up.t().contiguous()) * c
            dx[rows] += torch.mm(z, down)
            d_down[a, :q] = torch.mm(z.t().contiguous(), x[rows])
            d_up[a, :q] = torch.mm(h.t().contiguous(), dy[rows])
    return [out, dx, d_down, d_up] if train else out
