"""The measured cases of 4-bit weights and of mixtures of experts.

What a user keeps or serves beside a compressed FP8 layer:

  convert  values brought to microscaled 4-bit floating point (E2M1 in blocks of 32 with a power of two each) and back
  linear   the product with such a weight, of 16-bit activations or of activations in the same 4 bits
  grad     the gradient that a frozen 4-bit weight passes back to its input
  layer    a mixture-of-experts layer for a few tokens: the experts are chosen, their gated products computed and summed,
           with decoded E4M3 weights or 4-bit ones

`run` computes each in elementary torch operations, or, where `own` is set, through the package.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK, PITCH = 32, 128                     # values of one scale; stored rows are padded to this many values


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's activations: latency alone
        dict(name="convert_one_token", op="convert", rows=1, k=4096, x="bf16", to="bf16", pad=0),
        # the decoded gate projection of the 8192-wide block, taken from E4M3 to 4 bits
        dict(name="convert_weight", op="convert", rows=28672, k=8192, x="e4m3", to="bf16", pad=0),
        # one token of one request through a 4096-wide projection: latency alone
        dict(name="linear_one_token", op="linear", tokens=1, k=4096, n=4096, x="bf16", bias=False, pad=0),
        # a decode step of 45 requests in float16 at the 8192 to 28672 projection
        dict(name="linear_decode_45", op="linear", tokens=45, k=8192, n=28672, x="fp16", bias=False, pad=0),
        # a training batch's forward pass: activations keep 16 bits
        dict(name="linear_batch", op="linear", tokens=4096, k=8192, n=28672, x="bf16", bias=False, pad=0),
        # a prompt of odd length at the diffusion block's projection, an odd number of outputs, with a bias; 4-bit activations
        dict(name="mx_odd", op="linear", tokens=331, k=5120, n=13821, x="mx", bias=True, pad=64),
        # prompts with 4-bit activations, quantised in the pass
        dict(name="mx_prompts", op="linear", tokens=4096, k=8192, n=28672, x="mx", bias=False, pad=0),
        # a short odd sequence in training, float16
        dict(name="grad_77", op="grad", tokens=77, k=4096, n=14336, x="fp16"),
        # a training batch at the diffusion block's widest projection
        dict(name="grad_4096", op="grad", tokens=4096, k=5120, n=13824, x="bf16"),
        # one token through a layer of 256 experts, 8 of them chosen, weights decoded to E4M3
        dict(name="layer_one_token", op="layer", tokens=1, k=7168, inner=2048, experts=256, top=8, x="bf16", w="e4m3",
             score="softmax", bare=0.0),
        # a few requests, one of them padding, 8 experts of odd sizes, float16
        dict(name="layer_7_tokens", op="layer", tokens=7, k=4096, inner=1808, experts=8, top=2, x="fp16", w="e4m3",
             score="sigmoid", bare=0.15),
        # a decode step of 64 requests over 256 experts in 4 bits
        dict(name="layer_decode_64", op="layer", tokens=64, k=7168, inner=2048, experts=256, top=8, x="bf16", w="mx",
             score="softmax", bare=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["convert", "linear", "linear", "grad", "layer", "layer"])
    half = rng.choice(["bf16", "fp16"])
    if op == "convert":
        k = 32 * _log(rng, 1, 448)
        return dict(op=op, rows=_log(rng, 1, max(1, 100_000_000 // k)), k=k, x=rng.choice(["bf16", "fp16", "fp32", "e4m3"]),
                    to=rng.choice(["bf16", "fp32"]), pad=rng.choice([0, 0, 64, 8]))
    if op == "layer":
        k, inner = 32 * _log(rng, 1, 224), 32 * _log(rng, 1, 128)
        if rng.random() < 0.5:                                  # E4M3 weights come in multiples of 16
            w, k, inner = "e4m3", k - rng.choice([0, 16]), inner - rng.choice([0, 16])
        else:
            w = "mx"
        experts = _log(rng, 1, max(1, min(256, 1_500_000_000 // (3 * k * inner))))
        top = min(experts, rng.choice([1, 2, 4, 6, 8]))
        return dict(op=op, tokens=_log(rng, 1, 64), k=k, inner=inner, experts=experts, top=top, x=half, w=w,
                    score=rng.choice(["softmax", "sigmoid"]), bare=rng.choice([0.0, 0.0, 0.3]))
    k = 32 * _log(rng, 1, 448)
    n = _log(rng, 1, 14336)
    if op == "grad":
        n = max(8, n // 8 * 8)                                  # rows of dy on 16-byte borders
    most = 4096 * 8192 * 28672 // 4
    case = dict(op=op, tokens=_log(rng, 1, max(1, min(8192, most // (k * n)))), k=k, n=n, x=half)
    if op == "linear":
        case.update(x=rng.choice([half, "mx"]), bias=rng.random() < 0.4, pad=rng.choice([0, 0, 64, 8]))
    return case


# ------------------------------------------------------------------ inputs

def _quantised(v):
    """(…, K) float32 in blocks of 32: the rounded values over their scales, and the scales' exponents (…, K / 32)."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 3).clamp(min=-127)
    m = torch.ldexp(b, -e)
    a = m.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(a / step) * step).clamp(max=6), m)
    return q, e


def _packed(v):
    """(…, K) float32 as stored: two codes a byte, the first in the low half, and a byte for each block's exponent plus
    127; rows padded with zeros to a multiple of 128 values."""
    q, e = _quantised(v)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | torch.signbit(q).to(torch.uint8) << 3).reshape(v.shape)
    scales = (e[..., 0] + 127).to(torch.uint8)
    short = -v.shape[-1] % PITCH
    code = torch.nn.functional.pad(code, (0, short))
    scales = torch.nn.functional.pad(scales, (0, short // BLOCK))
    return code[..., 0::2] | code[..., 1::2] << 4, scales


def _weight(g, n, k, lead=()):
    """A weight as training leaves it, heavy tails included, float32."""
    w = torch.randn(*lead, n, k, generator=g, device="cuda")
    return w * (1 + 0.2 * w.square()) * (0.6 / math.sqrt(k))


def _spread(t, pad, g):
    """`t` as the leading columns of a wider buffer."""
    if not pad:
        return t
    wide = torch.randn(t.shape[0], t.shape[1] + pad, generator=g, device="cuda").to(t.dtype)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _activations(g, t, k):
    """Rows of different magnitude with a few large channels."""
    x = torch.randn(t, k, generator=g, device="cuda") * torch.exp(torch.randn(t, 1, generator=g, device="cuda") * 0.5)
    return x * torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 8.0, 1.0)


def _kept(packed, k):
    """The weight as the program keeps it."""
    if own:
        import lossless_entropy_coded_ecf8_amd as E
        return E.MXFP4(packed[0], packed[1], k)
    return packed


def prepare(case, seed):
    g, s = torch.Generator(device="cuda").manual_seed(seed), dict(case)
    if case["op"] == "convert":
        s["x_scale"] = None
        if case["x"] == "e4m3":
            x = _weight(g, case["rows"], case["k"])
            s["x_scale"] = x.abs().max() / 448
            x = (x / s["x_scale"]).to(torch.float8_e4m3fn)
        else:
            x = _activations(g, case["rows"], case["k"]).to(TYPES[case["x"]])
        s["values"] = _spread(x, case["pad"], g)
        return s
    if case["op"] == "layer":
        e, k, i = case["experts"], case["k"], case["inner"]
        s["values"] = _activations(g, case["tokens"], k).to(TYPES[case["x"]])
        s["logits"] = torch.randn(case["tokens"], e, generator=g, device="cuda") * 2
        rng = random.Random(seed)
        s["logits"][[t for t in range(case["tokens"]) if rng.random() < case["bare"]]] = -math.inf    # padding chooses none
        for name, rows, cols in (("gate", i, k), ("up", i, k), ("down", k, i)):
            if case["w"] == "mx":
                wide = -(-cols // PITCH) * PITCH
                codes = torch.empty(e, rows, wide // 2, dtype=torch.uint8, device="cuda")
                scales = torch.empty(e, rows, wide // BLOCK, dtype=torch.uint8, device="cuda")
                for j in range(e):
                    codes[j], scales[j] = _packed(_weight(g, rows, cols))
                s[name] = _kept((codes, scales), cols)
            else:
                s[name] = torch.empty(e, rows, cols, dtype=torch.uint8, device="cuda")
                s[name + "_scale"] = torch.empty(e, device="cuda")
                for j in range(e):
                    w = _weight(g, rows, cols)
                    s[name + "_scale"][j] = w.abs().max() / 448
                    s[name][j] = (w / s[name + "_scale"][j]).to(torch.float8_e4m3fn).view(torch.uint8)
        return s
    t, k, n = case["tokens"], case["k"], case["n"]
    s["w"] = _kept(_packed(_weight(g, n, k)), k)
    if case["op"] == "grad":
        s["dy"] = (torch.randn(t, n, generator=g, device="cuda") * 1e-2).to(TYPES[case["x"]])
        return s
    dt = TYPES["bf16" if case["x"] == "mx" else case["x"]]
    s["values"] = _spread(_activations(g, t, k).to(dt), case["pad"], g)
    s["shift"] = torch.randn(n, generator=g, device="cuda").to(dt) if case["bias"] else None
    return s


# ------------------------------------------------------------------ one pass

def _widened(packed, k):
    """The values of a stored weight, float32."""
    codes, scales = packed
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].reshape(*codes.shape[:-1], -1, BLOCK)
    return torch.ldexp(v, scales[..., None].int() - 127).reshape(*codes.shape[:-1], -1)[..., :k]


def _plain_layer(s):
    logits = s["logits"].float()
    best = torch.sort(logits, dim=1, descending=True, stable=True)
    values, ids = best.values[:, :s["top"]], best.indices[:, :s["top"]].int()
    score = torch.exp(values - logits.amax(1, keepdim=True)) if s["score"] == "softmax" else 1 / (1 + torch.exp(-values))
    here = values > -math.inf
    score = torch.where(here, score, 0.0)
    weights = torch.where(here, score / score.sum(1, keepdim=True), 0.0)
    ids = torch.where(here, ids, -1)
    x = s["values"].float()
    y = torch.zeros_like(x)
    for j in ids.unique().tolist():                             # each chosen expert's tokens in one product
        if j < 0:
            continue
        if s["w"] == "mx":
            gate, up, down = (_widened((s[w][0][j], s[w][1][j]), c) for w, c in
                              (("gate", s["k"]), ("up", s["k"]), ("down", s["inner"])))
        else:
            gate, up, down = (s[w][j].view(torch.float8_e4m3fn).float() * s[w + "_scale"][j] for w in ("gate", "up", "down"))
        t, c = (ids == j).nonzero(as_tuple=True)
        a = x[t] @ gate.t()
        h = a / (1 + torch.exp(-a)) * (x[t] @ up.t())
        y[t] += weights[t, c, None] * (h @ down.t())
    return [ids, weights, y.to(s["values"].dtype)]


def run(s):
    if own:
        import lossless_entropy_coded_ecf8_amd as E
        if s["op"] == "convert":
            return E.quantize_mxfp4(s["values"], s["x_scale"]).dequantize(TYPES[s["to"]])
        if s["op"] == "grad":
            return E.linear_mxfp4_input_grad(s["dy"], s["w"])
        if s["op"] == "linear":
            x = E.quantize_mxfp4(s["values"]) if s["x"] == "mx" else s["values"]
            return E.linear_mxfp4(x, s["w"], s["shift"])
        ids, weights = E.moe_route(s["logits"], s["top"], score=s["score"])
        if s["w"] == "mx":
            return [ids, weights, E.moe_few(s["values"], s["gate"], s["up"], s["down"], ids, weights)]
        return [ids, weights, E.moe_few(s["values"], s["gate"], s["up"], s["down"], ids, weights, gate_scale=s["gate_scale"],
                                        up_scale=s["up_scale"], down_scale=s["down_scale"])]
    if s["op"] == "layer":
        return _plain_layer(s)
    if s["op"] == "grad":
        return (s["dy"].float() @ _widened(s["w"], s["k"])).to(s["dy"].dtype)
    x = s["values"].float()
    if s["op"] == "convert":
        if s["x_scale"] is not None:
            x = x * s["x_scale"]
        return torch.ldexp(*_quantised(x)).reshape(x.shape).to(TYPES[s["to"]])
    if s["x"] == "mx":
        x = torch.ldexp(*_quantised(x)).reshape(x.shape)
    y = x @ _widened(s["w"], s["k"]).t()
    if s["shift"] is not None:
        y = y + s["shift"].float()
    return y.to(s["values"].dtype)


# ------------------------------------------------------------------ what it cannot do without

def work(case):
    k, size = case["k"], {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "mx": 2}
    four = 1 / 2 + 1 / BLOCK                                    # bytes of a value in 4 bits, its share of the scale included
    if case["op"] == "convert":
        m = case["rows"] * k
        return {"bytes": int(m * (size[case["x"]] + size[case["to"]])), "flops": 2 * m}
    if case["op"] == "layer":
        t, e, i, top = case["tokens"], case["experts"], case["inner"], case["top"]
        used = max(1, round(e * (1 - (1 - top / e) ** (t * (1 - case["bare"])))))       # experts that a batch is sure to meet
        return {"bytes": int(used * 3 * k * i * (four if case["w"] == "mx" else 1)) + 4 * t * (k + e + 2 * top),
                "flops": int(6 * t * (1 - case["bare"]) * top * k * i)}
    t, n = case["tokens"], case["n"]
    return {"bytes": int(n * k * four) + 2 * t * (k + n), "flops": 2 * t * n * k}


# ------------------------------------------------------------------ the definition in 64 bits

def _on_grid(m):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to each magnitude; half way, the one whose code is even."""
    code = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5))
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=m.device)[code]


def _through_4_bits(x):
    """Each block of 32 over the power of two that brings its largest magnitude into [4, 8), rounded, and back."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))), -125.0)
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))     # the logarithm's rounding
    unit = torch.exp2((e - 2).clamp(min=-127))
    return (torch.sign(b) * _on_grid(b.abs() / unit) * unit).reshape(x.shape)


def _from_bits(w, k):
    """The values of stored codes, from their bits: sign, 2 exponent bits of bias 1, 1 mantissa bit."""
    codes, scales = (w.data, w.scales) if own else w
    n = torch.arange(16, dtype=torch.float64, device=codes.device)
    e, m = torch.floor(n / 2) % 4, n % 2
    table = torch.where(n < 8, 1.0, -1.0) * torch.where(e == 0, m / 2, (1 + m / 2) * 2 ** (e - 1))
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    v[..., 0::2], v[..., 1::2] = table[(codes % 16).long()], table[(codes // 16).long()]
    return (v * (2.0 ** (scales.double() - 127)).repeat_interleave(BLOCK, -1))[..., :k]


def _e4m3_values():
    """The value of each E4M3 byte, from its bits: sign, 4 exponent bits of bias 7, 3 mantissa bits, no infinities."""
    got = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        got.append(math.nan if b & 127 == 127 else -v if b & 128 else v)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _exact_layer(s):
    logits = s["logits"].double().cpu().numpy()
    t, top = logits.shape[0], s["top"]
    ids, weights = np.full((t, top), -1, np.int32), np.zeros((t, top))
    for r in range(t):
        chosen = [c for c in np.lexsort((np.arange(logits.shape[1]), -logits[r]))[:top] if logits[r, c] > -np.inf]
        if chosen:
            v = logits[r, chosen]
            score = np.exp(v - v.max()) if s["score"] == "softmax" else 1 / (1 + np.exp(-v))
            ids[r, :len(chosen)], weights[r, :len(chosen)] = chosen, score / score.sum()
    x, table = s["values"].double(), _e4m3_values()
    y = torch.zeros_like(x)
    for j in sorted(set(ids.ravel().tolist()) - {-1}):
        part = []
        for w, c in (("gate", s["k"]), ("up", s["k"]), ("down", s["inner"])):
            if s["w"] == "mx":
                kept = s[w]
                codes, scales = (kept.data[j], kept.scales[j]) if own else (kept[0][j], kept[1][j])
                m = _from_bits(type(kept)(codes, scales, c) if own else (codes, scales), c)
            else:
                m = table[s[w][j].long()] * float(s[w + "_scale"][j])
            part.append(m.t().contiguous())
        rows, cols = np.nonzero(ids == j)
        at = torch.from_numpy(rows).cuda()
        a = torch.mm(x[at], part[0])
        h = a * torch.sigmoid(a) * torch.mm(x[at], part[1])
        y.index_add_(0, at, torch.from_numpy(weights[rows, cols]).cuda()[:, None] * torch.mm(h, part[2]))
    return [torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(), y]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        return _exact_layer(s)
    if case["op"] == "grad":
        return torch.mm(s["dy"].double(), _from_bits(s["w"], case["k"]))
    if case["op"] == "convert" and s["x_scale"] is not None:
        rows = [_through_4_bits((_e4m3_values()[v.view(torch.uint8).long()] * s["x_scale"].double()).float().double())
                for v in s["values"].split(1024)]               # the scaled value is a float32 by definition
        return torch.cat(rows)
    x = s["values"].double()
    if case["op"] == "convert":
        return _through_4_bits(x)
    y = torch.mm(_through_4_bits(x) if case["x"] == "mx" else x, _from_bits(s["w"], case["k"]).t().contiguous())
    return y if s["shift"] is None else y + s["shift"].double()
