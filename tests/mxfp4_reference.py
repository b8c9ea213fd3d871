"""Microscaled 4 bits and expert layers in 64 bits, and how far a kernel's result may be from them.

Conversion is exact: codes and scales have to be equal, values too.  Products, from the arithmetic: products of 16-bit
and widened values are exact in float32; a float32 sum of m terms is off by at most m 2^-23 of the sum of magnitudes; a
result is rounded once (bfloat16 2^-8, float16 2^-11 of the value, at least half of the smallest float16 step).
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def quantise(v):
    """(rows, K) float32 values on the CPU: codes (rows, K) and scale bytes (rows, K / 32)."""
    b = v.double().reshape(v.shape[0], -1, 32)
    m = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    e = torch.frexp(torch.where(bad, 1.0, m)).exponent - 1               # floor(log2 m)
    s = torch.where(m == 0, 0, (e - 2).clamp(min=-127) + 127)
    a = (b / torch.pow(2.0, (s - 127).double())[..., None]).abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    code = code + 8 * torch.signbit(b)
    code = torch.where(bad[..., None], 0, code)
    return code.reshape(v.shape).to(torch.uint8), torch.where(bad, 255, s).to(torch.uint8)


def store(code, scale):
    """As stored: rows padded with zeros to 128 values, two codes a byte."""
    short = -code.shape[-1] % 128
    code = torch.nn.functional.pad(code, (0, short))
    return code[..., 0::2] | code[..., 1::2] << 4, torch.nn.functional.pad(scale, (0, short // 32))


def values(data, scales, K):
    """The stored values in float64, on the CPU."""
    data, scales = data.cpu(), scales.cpu()
    code = torch.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], -1)
    unit = torch.where(scales == 255, torch.nan, torch.pow(2.0, scales.double() - 127))
    return (VALUES[code.long()] * unit.repeat_interleave(32, -1))[..., :K]


def random_stored(lead, K, g, lo=110, hi=128):
    """Random codes and scale bytes in [lo, hi), as stored."""
    code = torch.randint(0, 16, (*lead, K), generator=g).to(torch.uint8)
    scale = torch.randint(lo, hi, (*lead, K // 32), generator=g).to(torch.uint8)
    return store(code, scale)


def rounded(ref, err, dtype):
    return err + HALF[dtype] * (ref.abs() + err) + TINY[dtype]


def product(a, b, dtype, shift=None):
    """a b^T + shift in float64 and a kernel's tolerance."""
    ref, mag = a @ b.t(), a.abs() @ b.abs().t()
    if shift is not None:
        ref, mag = ref + shift, mag + shift.abs()
    return ref, rounded(ref, mag * (a.shape[1] + 8) * 2.0 ** -23, dtype)


def check(got, ref, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), what
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    worst = ((got - ref).abs() - tol)[fine]
    assert worst.numel() == 0 or float(worst.max()) <= 0, (what, float(worst.max()), float((got - ref)[fine].abs().max()))


def layer(x, gate, up, down, ids, weights, dtype):
    """y of an expert layer (weights as float64 stacks) and a kernel's tolerance: a and b are float32 sums; exp, the
    division and the products around them are off by at most 2^-20 of h together (the exponential 2 ulp, its argument
    exact to the error of a); h enters the second sum with 2^-16; a token's sum adds its choices."""
    T, top = ids.shape
    y = torch.zeros(T, x.shape[1], dtype=torch.float64)
    err = torch.zeros_like(y)
    for t in range(T):
        for j in range(top):
            e = int(ids[t, j])
            if not 0 <= e < gate.shape[0]:
                continue
            eps = (x.shape[1] + 8) * 2.0 ** -23
            a, b = gate[e] @ x[t], up[e] @ x[t]
            da, db = (gate[e].abs() @ x[t].abs()) * eps, (up[e].abs() @ x[t].abs()) * eps
            silu = a * torch.sigmoid(a)
            h = silu * b
            dh = 1.1 * da * (b.abs() + db) + silu.abs() * db + h.abs() * (2.0 ** -16 + 2.0 ** -20)    # |silu'| < 1.1
            w = float(weights[t, j])
            part = w * (down[e] @ h)
            mag = abs(w) * (down[e].abs() @ (h.abs() + dh))
            y[t] += part
            err[t] += abs(w) * (down[e].abs() @ dh) + mag * (down.shape[2] + top + 16) * 2.0 ** -23
    return y, rounded(y, err, dtype)
