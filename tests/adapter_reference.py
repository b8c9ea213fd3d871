"""The adapters' formulas in 64 bits, and how far a kernel's result may be from them.

Kernel error, from the arithmetic: products of 16-bit (or E4M3) values are
exact in float32; a float32 sum of m terms is off by at most m 2^-23 of the sum
of magnitudes; h and z enter their second product as two bfloat16 (2^-16 of
the value) and the float16 operands as two exact bfloat16, whose smallest cross
term is dropped (2^-16 more); the result is rounded once (bfloat16 2^-8,
float16 2^-11 of the value, at least half of the smallest float16 step).
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}


def part(v, f, g, scale, inner):
    """((v f^T) scale) g and its largest error before the final rounding, for inner + rank terms summed in float32."""
    low = (v @ f.t()) * scale
    low_mag = (v.abs() @ f.abs().t()) * abs(scale)
    eps = 2.0 ** -15 + (inner + f.shape[0] + 8) * 2.0 ** -23
    return low, low_mag, low @ g, (low_mag @ g.abs()) * eps


def rounded(ref, err, dtype):
    return err + HALF[dtype] * (ref.abs() + err) + TINY[dtype]


def adapters(base, x, x_scale, down, up, scaling, index, ranks, dy=None, dx_base=None):
    """dict of (reference, tolerance) in float64 on the CPU: out and, with dy, dx, d_down, d_up."""
    dt = down.dtype
    L, R, K = down.shape
    N = up.shape[2]
    d = lambda t: t.detach().to(torch.float32).cpu().double()  # noqa: E731
    x, down, up, scaling, index = d(x), d(down), d(up), d(scaling), index.cpu().long()
    T = index.numel()
    if x_scale is not None:
        x = x * float(x_scale)
    out = d(base) if base is not None else torch.zeros(T, N, dtype=torch.float64)
    oerr = torch.zeros_like(out)
    res = {}
    if dy is not None:
        dy = d(dy)
        dx = d(dx_base) if dx_base is not None else torch.zeros(T, K, dtype=torch.float64)
        derr = torch.zeros_like(dx)
        gd, ge = torch.zeros_like(down), torch.zeros_like(down)
        hd, he = torch.zeros_like(up), torch.zeros_like(up)
    for a in range(L):
        rows = (index == a).nonzero()[:, 0]
        q = R if ranks is None else max(0, min(R, int(ranks[a])))
        f, g, c = down[a, :q], up[a, :q], float(scaling[a])
        h, h_mag, o, e = part(x[rows], f, g, c, K)
        out[rows] += o
        oerr[rows] += e
        if dy is not None:
            z, z_mag, o, e = part(dy[rows], g, f, c, N)
            dx[rows] += o
            derr[rows] += e
            eps = 2.0 ** -15 + (K + N + rows.numel() + 8) * 2.0 ** -23
            gd[a, :q], ge[a, :q] = z.t() @ x[rows], (z_mag.t() @ x[rows].abs()) * eps
            hd[a, :q], he[a, :q] = h.t() @ dy[rows], (h_mag.t() @ dy[rows].abs()) * eps
    res["out"] = (out, rounded(out, oerr, dt))
    if dy is not None:
        res["dx"] = (dx, rounded(dx, derr, dt))
        res["d_down"] = (gd, rounded(gd, ge, dt))
        res["d_up"] = (hd, rounded(hd, he, dt))
    return res


def check(got, ref_tol, what=""):
    ref, tol = ref_tol
    got = got.detach().float().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), what
    worst = ((got - ref).abs() - tol).max() if got.numel() else torch.tensor(-1.0)
    assert float(worst) <= 0, (what, float(worst), float((got - ref).abs().max()))
