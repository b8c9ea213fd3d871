"""The entry points of include/ecf8a.h without a GPU: what they refuse, and the sizes they ask for.

Every call here is refused before anything is launched, so that the pointers, which point nowhere, are not followed.
"""
import ctypes
import os
import re

import pytest

import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import adapters as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 40                                                       # an aligned address that is never read
ARG, SIZE, UNSUPPORTED, WORKSPACE = -1, -2, -4, -7


def plan(tokens=100, adapters=4):
    return A.PlanA(P, 1 << 40, tokens, adapters, 160, 6, 4, 256)


def bank(**k):
    f = dict(down=P, up=P, scaling=P, ranks=None, in_features=64, out_features=48, adapters=4, rank=8, type=1, reserved=0)
    f.update(k)
    return A.BankA(*[f[n] for n, _ in A.BankA._fields_])


def test_every_declared_function_is_exported():
    src = open(os.path.join(ROOT, "include", "ecf8a.h")).read()
    names = set(re.findall(r"^(?:int|uint64_t) (ecf8a_\w+)\(", src, re.M))
    assert names == set(A.EXPORTS_A)
    lib = E.lib()
    for n in names:
        assert hasattr(lib, n)


def test_plan_bytes_and_refusals():
    L = A._lib()
    assert L.ecf8a_plan_bytes(0, 1) > 0 and L.ecf8a_plan_bytes(1 << 24, 2048) > 4 << 24
    for tokens, adapters in ((1, 0), (1, 2049), ((1 << 24) + 1, 1)):
        assert L.ecf8a_plan_bytes(tokens, adapters) == 0
    c = A.PlanA()
    call = lambda index=P, size=4, tokens=10, adapters=2, ws=P, n=1 << 30: L.ecf8a_plan_prepare(  # noqa: E731
        index, size, tokens, adapters, ws, n, None, ctypes.byref(c))
    for rc, k in ((ARG, dict(index=None)), (ARG, dict(index=P + 2)), (ARG, dict(index=P + 4, size=8)), (ARG, dict(size=2)),
                  (SIZE, dict(adapters=0)), (SIZE, dict(adapters=5000)), (SIZE, dict(tokens=1 << 25)), (WORKSPACE, dict(ws=None)),
                  (WORKSPACE, dict(ws=P + 16)), (WORKSPACE, dict(n=64))):
        assert call(**k) == rc, k
    assert L.ecf8a_plan_prepare(P, 4, 10, 2, P, 1 << 30, None, None) == ARG


@pytest.mark.parametrize("few", [False, True])
def test_add_refusals(few):
    L = A._lib()

    def call(b=None, p=None, x=P, ldx=64, xt=1, xs=None, base=P, ldb=48, out=P + 4096, ldo=48, hidden=None, ws=P, n=1 << 40, **k):
        b = bank(**k) if b is None else b
        if few:
            return L.ecf8a_add_few(P, 4, 100, ctypes.byref(b), x, ldx, xt, xs, base, ldb, out, ldo, ws, n, None)
        q = plan() if p is None else p
        return L.ecf8a_add(ctypes.byref(q), ctypes.byref(b), x, ldx, xt, xs, base, ldb, out, ldo, hidden, ws, n, None)

    big = dict(in_features=65536, out_features=48)                # too large for one kernel: a workspace is needed
    for rc, k in ((UNSUPPORTED, dict(type=3)), (UNSUPPORTED, dict(type=0)), (UNSUPPORTED, dict(xt=2)), (SIZE, dict(rank=0)),
                  (SIZE, dict(rank=257)), (SIZE, dict(in_features=0)), (SIZE, dict(out_features=(1 << 20) + 1)),
                  (SIZE, dict(adapters=0)), (SIZE, dict(adapters=2049)), (ARG, dict(down=None)), (ARG, dict(up=P + 1)),
                  (ARG, dict(scaling=P + 2)), (ARG, dict(ranks=P + 1)), (ARG, dict(x=None)), (ARG, dict(out=None)),
                  (ARG, dict(x=P + 1)), (ARG, dict(base=P + 1)), (ARG, dict(xs=P + 2)), (ARG, dict(base=P, out=P, ldo=50)),
                  (SIZE, dict(ldx=63)), (SIZE, dict(ldb=47)), (SIZE, dict(ldo=47)),
                  (WORKSPACE, dict(ws=None, ldx=65536, **big)), (WORKSPACE, dict(ws=P + 8, ldx=65536, **big)),
                  (WORKSPACE, dict(n=300, ldx=65536, **big))):  # 300 bytes: below any need
        assert call(**k) == rc, k
    if few:
        assert call(rank=65) == SIZE
        assert L.ecf8a_add_few(P, 4, 513, ctypes.byref(bank()), P, 64, 1, None, P, 48, P, 48, P, 1 << 30, None) == SIZE
        assert L.ecf8a_add_few(P, 3, 5, ctypes.byref(bank()), P, 64, 1, None, P, 48, P, 48, P, 1 << 30, None) == ARG
        assert L.ecf8a_add_few(None, 4, 5, ctypes.byref(bank()), P, 64, 1, None, P, 48, P, 48, P, 1 << 30, None) == ARG
        assert L.ecf8a_add_few(None, 4, 0, ctypes.byref(bank()), None, 64, 1, None, None, 0, None, 48, None, 0, None) == 0
        assert L.ecf8a_few(512, ctypes.byref(bank())) == 1 and L.ecf8a_few(513, ctypes.byref(bank())) == 0
        assert L.ecf8a_few(1, ctypes.byref(bank(rank=65))) == 0 and L.ecf8a_few(1, None) == 0
    else:
        assert call(p=plan(adapters=5)) == ARG and call(p=plan(adapters=0)) == ARG and call(hidden=P + 8) == ARG
        assert call(p=plan(tokens=0), x=None, out=None, ws=None) == 0


def test_grads_refusals():
    L = A._lib()

    def call(p=None, dy=P, ldy=48, x=P, ldx=64, hidden=None, dxb=None, ldb=0, dx=P + 8192, ldd=64, dd=P, du=P, ws=P, n=1 << 50, **k):
        q = plan() if p is None else p
        return L.ecf8a_grads(ctypes.byref(q), ctypes.byref(bank(**k)), dy, ldy, x, ldx, hidden, dxb, ldb, dx, ldd, dd, du, ws, n, None)

    for rc, k in ((UNSUPPORTED, dict(type=4)), (ARG, dict(dd=None)), (ARG, dict(du=P + 1)), (ARG, dict(dy=None)), (ARG, dict(x=None)),
                  (ARG, dict(hidden=P + 4)), (ARG, dict(dxb=P, dx=P, ldb=66)), (SIZE, dict(ldy=47)), (SIZE, dict(ldx=60)),
                  (SIZE, dict(ldd=63)), (SIZE, dict(dxb=P + 64, ldb=3)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(n=512)),
                  (ARG, dict(adapters=3)), (SIZE, dict(rank=300))):
        assert call(**k) == rc, k


def test_input_grad_refusals_and_sizes():
    L = A._lib()

    def call(dy=P, ldy=64, T=10, N=64, w=P, K=32, s=P, t=1, dx=P, ldx=32, ws=P, n=1 << 40):
        return L.ecf8a_input_grad(dy, ldy, T, N, w, K, s, t, dx, ldx, ws, n, None)

    for rc, k in ((UNSUPPORTED, dict(t=3)), (UNSUPPORTED, dict(t=4)), (SIZE, dict(N=72)), (SIZE, dict(K=40)), (SIZE, dict(N=0)),
                  (SIZE, dict(T=1 << 25)), (ARG, dict(dy=None)), (ARG, dict(w=P + 8)), (ARG, dict(s=P + 1)), (ARG, dict(dx=P + 2)),
                  (ARG, dict(ldy=65)), (ARG, dict(ldx=36)), (SIZE, dict(ldy=56)), (SIZE, dict(ldx=24)), (SIZE, dict(ldy=1 << 23)),
                  (WORKSPACE, dict(N=65536, ldy=65536, ws=None)), (WORKSPACE, dict(N=65536, ldy=65536, n=16))):
        assert call(**k) == rc, k
    assert call(T=0, dy=None, w=None, dx=None) == 0
    assert L.ecf8a_input_grad_bytes(10, 65536, 32) > 0 and L.ecf8a_input_grad_bytes(4096, 4096, 4096) == 0
    assert L.ecf8a_input_grad_bytes(10, 17, 32) == 0


def test_clip_refusals():
    L = A._lib()
    c = A.ClipPlanA()

    def call(rows, type_=3, ws=P, n=1 << 40):
        arr = (A.GradA * max(1, len(rows)))(*[A.GradA(*r) for r in rows])
        return L.ecf8a_clip_prepare(arr, len(rows), type_, ws, n, None, ctypes.byref(c))

    for rc, rows, k in ((UNSUPPORTED, [(P, P, 4)], dict(type_=4)), (ARG, [(None, P, 4)], {}), (ARG, [(P, None, 4)], {}),
                        (ARG, [(P + 2, P + 2, 4)], {}), (ARG, [(P, P + 2, 4)], {}), (ARG, [(P, P, 8), (P + 16, P + 16, 8)], {}),
                        (ARG, [(P, P + 16, 8)], {}), (ARG, [(P, P, 8), (P, P, 8)], {}), (ARG, [(P, P + 64, 8), (P + 128, P + 64, 8)], {}),
                        (SIZE, [(P, P, 1 << 41)], {}), (WORKSPACE, [(P, P, 8)], dict(ws=None)), (WORKSPACE, [(P, P, 8)], dict(ws=P + 64)),
                        (WORKSPACE, [(P, P, 8)], dict(n=1024))):
        assert call(rows, **k) == rc, (rows, k)
    assert L.ecf8a_clip_bytes(None, 3) == 0 and L.ecf8a_clip_bytes(None, 0) > 0
    good = A.ClipPlanA(P, 1 << 20, 1, 1, 3, 1, 1)
    for bad, norm in ((-1.0, P), (float("nan"), P), (1.0, None), (1.0, P + 2)):
        assert L.ecf8a_clip_run(ctypes.byref(good), bad, norm, None) == ARG
    assert L.ecf8a_clip_run(ctypes.byref(A.ClipPlanA(None, 0, 1, 1, 3, 1, 1)), 1.0, P, None) == ARG
    assert L.ecf8a_clip_run(ctypes.byref(A.ClipPlanA(P, 0, 1, 1, 3, 0, 1)), 1.0, P, None) == ARG
    assert L.ecf8a_clip_run(ctypes.byref(A.ClipPlanA(P, 0, 1, 1, 9, 1, 1)), 1.0, P, None) == ARG
