"""The entry points of include/ecf8x.h and their Python forms without a GPU: what they refuse, and the sizes they ask for.

Every call here is refused before anything is launched, so that the pointers, which point nowhere, are not followed.
"""
import ctypes
import os
import re

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import mxfp4 as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 40                                                       # an aligned address that is never read
ARG, SIZE, UNSUPPORTED, WORKSPACE = -1, -2, -4, -7


def matrix(codes=P, scales=P, factors=None):
    return M.MatrixX(codes, scales, factors)


def test_every_declared_function_is_exported():
    src = open(os.path.join(ROOT, "include", "ecf8x.h")).read()
    names = set(re.findall(r"^(?:int|uint64_t) (ecf8x_\w+)\(", src, re.M))
    assert names == set(M.EXPORTS_X)
    lib = E.lib()
    for n in names:
        assert hasattr(lib, n)


def test_conversion_refusals():
    L = M._lib()
    q = lambda x=P, ld=64, t=1, s=None, rows=3, cols=64, c=P, sc=P: L.ecf8x_quantize(x, ld, t, s, rows, cols, c, sc, None)  # noqa: E731
    for rc, k in ((UNSUPPORTED, dict(t=0)), (UNSUPPORTED, dict(t=5)), (SIZE, dict(cols=0)), (SIZE, dict(cols=48)), (SIZE, dict(cols=1 << 21)),
                  (SIZE, dict(rows=1 << 31)), (SIZE, dict(ld=63)), (ARG, dict(x=None)), (ARG, dict(c=None)), (ARG, dict(sc=None)),
                  (ARG, dict(x=P + 1)), (ARG, dict(t=3, x=P + 2)), (ARG, dict(c=P + 8)), (ARG, dict(sc=P + 2)), (ARG, dict(s=P)),
                  (ARG, dict(t=4, s=P + 2))):
        assert q(**k) == rc, k
    assert q(rows=0, x=None) == 0
    d = lambda c=P, s=P, rows=3, cols=64, t=1, out=P, ld=64: L.ecf8x_dequantize(c, s, rows, cols, t, out, ld, None)  # noqa: E731
    for rc, k in ((UNSUPPORTED, dict(t=4)), (SIZE, dict(cols=33)), (SIZE, dict(ld=56)), (ARG, dict(ld=65)), (ARG, dict(out=P + 8)),
                  (ARG, dict(c=None)), (ARG, dict(s=P + 1))):
        assert d(**k) == rc, k
    assert d(rows=0, c=None) == 0


def test_product_refusals():
    L = M._lib()

    def call(x=P, xs=None, ldx=64, xt=1, T=3, N=5, K=64, w=matrix(), b=None, yt=1, y=P, ldy=5, ws=None, n=0):
        return L.ecf8x_linear(x, xs, ldx, xt, T, N, K, None if w is None else ctypes.byref(w), b, yt, y, ldy, ws, n, None)

    for rc, k in ((UNSUPPORTED, dict(xt=3, yt=3)), (UNSUPPORTED, dict(xt=1, yt=2)), (UNSUPPORTED, dict(xt=4)), (UNSUPPORTED, dict(xt=5, yt=3)),
                  (SIZE, dict(N=0)), (SIZE, dict(K=48)), (SIZE, dict(K=0)), (SIZE, dict(T=1 << 25)), (SIZE, dict(N=1 << 21)), (SIZE, dict(ldx=56)),
                  (SIZE, dict(ldx=1 << 23)), (SIZE, dict(ldy=4)), (ARG, dict(x=None)), (ARG, dict(x=P + 8)), (ARG, dict(ldx=65)), (ARG, dict(xs=P)),
                  (ARG, dict(xt=5, xs=None)), (ARG, dict(xt=5, xs=P + 2)), (ARG, dict(w=None)), (ARG, dict(w=matrix(None))), (ARG, dict(w=matrix(P + 8))),
                  (ARG, dict(w=matrix(P, None))), (ARG, dict(w=matrix(P, P + 1))), (ARG, dict(y=None)), (ARG, dict(y=P + 1)), (ARG, dict(b=P + 1))):
        assert call(**k) == rc, k
    assert call(T=0, x=None) == 0
    big = dict(T=100, N=64, K=65536, ldx=65536, ldy=64)
    need = L.ecf8x_linear_bytes(100, 64, 65536, 1)
    assert need >= 2 * 4 * 100 * 64 and need % 256 == 0
    for k in (dict(ws=None), dict(ws=P + 16, n=1 << 40), dict(ws=P, n=need - 1)):
        assert call(**big, **k) == WORKSPACE
    for sizes in ((1, 28672, 8192), (64, 28672, 8192), (100, 64, 48), (100, 0, 64)):
        assert L.ecf8x_linear_bytes(*sizes, 1) == 0

    def grad(dy=P, ld=64, t=1, T=3, N=64, K=64, w=matrix(), dx=P, ldx=64, ws=None, n=0):
        return L.ecf8x_input_grad(dy, ld, t, T, N, K, None if w is None else ctypes.byref(w), dx, ldx, ws, n, None)

    for rc, k in ((UNSUPPORTED, dict(t=5)), (SIZE, dict(K=40)), (SIZE, dict(N=0)), (SIZE, dict(ld=56)), (SIZE, dict(ldx=56)), (SIZE, dict(ld=1 << 23)),
                  (ARG, dict(dy=None)), (ARG, dict(dy=P + 2)), (ARG, dict(dx=P + 8)), (ARG, dict(ld=65)), (ARG, dict(ldx=66)), (ARG, dict(w=None)),
                  (ARG, dict(w=matrix(P + 1))), (WORKSPACE, dict(T=40, N=65536, ld=65536))):
        assert grad(**k) == rc, k
    assert grad(T=0, dy=None) == 0


def layer(four=False, **k):
    m = matrix() if four else matrix(P, None, P)
    f = dict(gate=m, up=m, down=m, features=64, inner=96, experts=4, type=5 if four else 4)
    f.update(k)
    return M.ExpertsX(*[f[n] for n, _ in M.ExpertsX._fields_])


def test_expert_refusals():
    L = M._lib()
    r = lambda x=P, ld=8, t=3, T=3, e=8, top=2, s=0, n=1, i=P, w=P: L.ecf8x_route(x, ld, t, T, e, top, s, n, 1.0, i, w, None)  # noqa: E731
    for rc, k in ((UNSUPPORTED, dict(t=4)), (UNSUPPORTED, dict(s=2)), (SIZE, dict(e=0)), (SIZE, dict(e=1025, ld=2000)), (SIZE, dict(top=0)),
                  (SIZE, dict(top=9)), (SIZE, dict(e=64, ld=64, top=33)), (SIZE, dict(ld=7)), (ARG, dict(x=None)), (ARG, dict(x=P + 2)),
                  (ARG, dict(i=P + 2)), (ARG, dict(w=None))):
        assert r(**k) == rc, k
    assert r(T=0, x=None) == 0

    def call(l=None, x=P, ldx=64, t=1, T=3, top=2, i=P, w=P, y=P, ldy=64, ws=P, n=1 << 30, **k):
        q = layer(**k) if l is None else l
        return L.ecf8x_moe(x, ldx, t, T, top, i, w, ctypes.byref(q), y, ldy, ws, n, None)

    for four in (False, True):
        for rc, k in ((UNSUPPORTED, dict(t=3)), (UNSUPPORTED, dict(type=1)), (SIZE, dict(features=72)), (SIZE, dict(inner=0)), (SIZE, dict(inner=1 << 17)),
                      (SIZE, dict(experts=0)), (SIZE, dict(experts=1025)), (SIZE, dict(top=0)), (SIZE, dict(top=33)), (SIZE, dict(T=257)),
                      (SIZE, dict(ldx=56)), (SIZE, dict(ldy=63)), (ARG, dict(x=None)), (ARG, dict(x=P + 8)), (ARG, dict(ldx=65)), (ARG, dict(i=None)),
                      (ARG, dict(w=P + 2)), (ARG, dict(y=P + 1)), (ARG, dict(gate=matrix(None))), (ARG, dict(up=matrix(P, P + 1))),
                      (ARG, dict(down=matrix(P + 4, None))), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=P + 8)), (WORKSPACE, dict(n=100))):
            assert call(four=four, **k) == rc, (four, k)
    assert call(gate=matrix(P, P)) == ARG and call(four=True, up=matrix(P, P, P)) == ARG and call(inner=112, n=0) == WORKSPACE
    assert call(four=True, inner=112) == SIZE
    assert call(T=0, x=None) == 0
    l = layer()
    assert L.ecf8x_moe_bytes(3, 2, ctypes.byref(l)) >= 3 * 2 * 4 * 96 and L.ecf8x_moe_bytes(257, 2, ctypes.byref(l)) == 0
    assert L.ecf8x_moe_bytes(3, 2, None) == 0
    assert L.ecf8x_moe(P, 64, 1, 3, 2, P, P, None, P, 64, P, 1 << 30, None) == ARG


def four(*lead, k=64, device="cpu"):
    wide = -(-k // 128) * 128
    return E.MXFP4(torch.zeros(*lead, wide // 2, dtype=torch.uint8, device=device), torch.zeros(*lead, wide // 32, dtype=torch.uint8, device=device), k)


def test_stored_form_is_checked():
    u8 = torch.uint8
    for data, scales, k in ((torch.zeros(3, 64, dtype=u8), torch.zeros(3, 4, dtype=u8), 48), (torch.zeros(3, 32, dtype=u8), torch.zeros(3, 4, dtype=u8), 64),
                            (torch.zeros(3, 64, dtype=u8), torch.zeros(3, 2, dtype=u8), 64), (torch.zeros(3, 64), torch.zeros(3, 4, dtype=u8), 64),
                            (torch.zeros(3, 64, dtype=u8), torch.zeros(2, 4, dtype=u8), 64), (torch.zeros(64, dtype=u8), torch.zeros(4, dtype=u8), 64),
                            (torch.zeros(3, 128, dtype=u8)[:, :64], torch.zeros(3, 4, dtype=u8), 64),
                            (torch.zeros(3 * 64 + 8, dtype=u8)[8:].view(3, 64), torch.zeros(3, 4, dtype=u8), 64)):
        with pytest.raises(ValueError):
            E.MXFP4(data, scales, k)
    q = four(3, 5, k=96)
    assert q.shape == (3, 5, 96) and q.nbytes() == 15 * 68


def test_calls_off_the_gpu_or_of_other_shapes_are_refused():
    x, w = torch.zeros(3, 64, dtype=torch.bfloat16), four(5)
    for call in (lambda: E.quantize_mxfp4(x), lambda: w.dequantize(), lambda: w.dequantize(torch.float64), lambda: E.linear_mxfp4(x, w),
                 lambda: E.linear_mxfp4_input_grad(x, w), lambda: E.moe_route(torch.zeros(3, 4), 2),
                 lambda: E.moe_few(x, four(2, 32), four(2, 32), four(2, 64, k=32), torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, 1)),
                 lambda: E.linear_mxfp4(x, four(2, 5))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        E.linear_mxfp4(x, torch.zeros(5, 64))


def test_calls_that_keep_no_gradients_say_so_once(monkeypatch):
    import warnings
    monkeypatch.setattr(M, "_warned", set())
    w = four(5)
    calls = {"linear_mxfp4": lambda x: E.linear_mxfp4(x, w), "moe_route": lambda x: E.moe_route(x, 2),
             "moe_few": lambda x: E.moe_few(x, w, w, w, torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, 1))}
    for name, call in calls.items():
        for grad, heard in ((False, 0), (True, 1), (True, 0)):
            with warnings.catch_warnings(record=True) as got:
                warnings.simplefilter("always")
                with pytest.raises(ValueError):                   # not on a GPU
                    call(torch.zeros(3, 64, dtype=torch.bfloat16).requires_grad_(grad))
            assert len(got) == heard and all(name in str(m.message) for m in got), name
