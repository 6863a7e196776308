"""The row operators without a GPU: their 64-bit forms against differences, and
the host checks of every entry point (bad arguments are refused before
anything is launched; the pointers here are never dereferenced)."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import mixture_experts_layer_07_amd as moe
import rowops_ref as ref
from mixture_experts_layer_07_amd import binding

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
ODD = C.c_void_p((1 << 20) + 4)
A, B, D, E, F, G, I, J, K = (C.c_void_p(n << 24) for n in range(1, 10))  # buffers, never dereferenced
F32, BF16, FP8 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from mixture_experts_layer_07_amd import build
        build.build(verbose=False)
    return moe.lib()


# ------------------------------------------------- formulas against differences
def rnd(*shape, seed=0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape))


def close(a, b, tol):
    assert abs(a - b) <= tol * max(1.0, abs(b)), (a, b)


def test_rmsnorm_formula():
    z, w, dy, v, u = rnd(5, 24), 1 + 0.1 * rnd(24, seed=1), rnd(5, 24, seed=2), rnd(5, 24, seed=3), rnd(24, seed=4)
    dz, dw, _, _ = ref.rmsnorm_backward(dy, z, w, 1e-3)
    close(ref.differences(lambda a: (ref.rmsnorm(a, w, 1e-3) * dy).sum(), z, v, 1e-5), float((dz * v).sum()), 1e-8)
    close(ref.differences(lambda a: (ref.rmsnorm(z, a, 1e-3) * dy).sum(), w, u, 1e-5), float((dw * u).sum()), 1e-8)
    both, _, _, _ = ref.rmsnorm_backward(dy, z, w, 1e-3, v)
    assert torch.allclose(both, dz + v, rtol=0, atol=1e-14)


def test_finalize_formula():
    T, k, H, sh = 6, 3, 8, 2
    up = torch.randperm(T * k, generator=torch.Generator().manual_seed(0)).int()
    fc2, sc, dy = rnd(T * (k + sh), H), rnd(T, k, seed=1), rnd(T, H, seed=2)
    vf, vs = rnd(*fc2.shape, seed=3), rnd(T, k, seed=4)
    # the weighted rows' gradient is dispatch of scaled dy; with scales 1 its transpose is dispatch_backward
    df = ref.dispatch(dy, up, k, sh)
    df[up.long()] *= sc.reshape(-1, 1)
    close(ref.differences(lambda a: (ref.finalize(a, up, sc, sh) * dy).sum(), fc2, vf, 1e-4), float((df * vf).sum()), 1e-8)
    ds = (fc2[up.long()].view(T, k, H) * dy[:, None]).sum(2)
    close(ref.differences(lambda a: (ref.finalize(fc2, up, a, sh) * dy).sum(), sc, vs, 1e-4), float((ds * vs).sum()), 1e-8)
    dx, _ = ref.dispatch_backward(fc2, up, k, sh)
    close(ref.differences(lambda a: (ref.dispatch(a, up, k, sh) * fc2).sum(), dy, rnd(T, H, seed=5), 1e-4),
          float((dx * rnd(T, H, seed=5)).sum()), 1e-8)
    assert torch.allclose(dx, ref.finalize(fc2, up, torch.ones(T, k), sh), rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("method", range(7))
def test_route_formula(method, renorm):
    T, E, k = 7, 11, 4
    l, ds, v = rnd(T, E), rnd(T, k, seed=1), rnd(T, E, seed=2)
    ids = l.topk(k, 1).indices.int()
    d, size = ref.route_backward(l, ids, ds, method, 2.5, renorm)
    f = lambda a: (ref.route_scales(a, ids, method, 2.5, renorm) * ds).sum()  # noqa: E731
    close(ref.differences(f, l, v, 1e-5), float((d * v).sum()), 1e-8)
    assert (d.abs() <= size * (1 + 1e-12)).all()


def test_swiglu_formula():
    gu, dh, v = rnd(5, 32), rnd(5, 16, seed=1), rnd(5, 32, seed=2)
    d, size = ref.swiglu_backward(dh, gu)
    close(ref.differences(lambda a: (ref.swiglu(a) * dh).sum(), gu, v, 1e-5), float((d * v).sum()), 1e-8)
    assert (d.abs() <= size * (1 + 1e-12)).all()


# ------------------------------------------------------------------- refusals
def test_rmsnorm_validation(L):
    def f(x=A, r=None, w=B, dt=BF16, T=4, H=256, eps=1e-6, total=None, y=D, q=None, s=None):
        return L.moe_rmsnorm(x, r, w, dt, T, H, eps, total, y, q, s, None)

    assert f(T=-1) == INVALID and f(H=0) == INVALID and f(dt=FP8) == INVALID and f(dt=7) == INVALID
    assert f(H=100) == UNSUPPORTED                          # H % 8
    assert f(H=16392) == UNSUPPORTED and "16384" in binding.last_error()
    assert f(T=(1 << 30) + 1) == UNSUPPORTED
    assert f(H=264, q=E, s=F) == UNSUPPORTED                # codes need H % 128
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert f(eps=eps) == INVALID
    assert f(x=None) == INVALID and f(w=None) == INVALID
    assert f(r=E) == INVALID and f(total=E) == INVALID      # residual and total together
    assert f(q=E) == INVALID and f(s=E) == INVALID          # codes and scales together
    assert f(y=None) == INVALID                             # nothing to write
    full = dict(x=A, r=E, w=B, total=F, y=D, q=G, s=I)
    for out, others in (("y", ("total", "r", "w", "q", "s")), ("total", ("w", "q", "s")), ("q", ("x", "r", "w", "s")),
                        ("s", ("x", "r", "w"))):
        for other in others:
            assert f(**{**full, out: full[other]}) == INVALID and "same buffer" in binding.last_error()
    for name in ("x", "r", "w", "total", "y", "q"):
        a = dict(full)
        a[name] = ODD
        assert f(**a) == INVALID and "aligned" in binding.last_error()
    assert f(x=None, w=None, y=None, T=0) == OK


def test_rmsnorm_backward_validation(L):
    def f(dy=A, z=B, w=D, d=None, dt=BF16, T=4, H=256, eps=1e-6, dz=E, dw=F, ws=G, n=1 << 30):
        return L.moe_rmsnorm_backward(dy, z, w, d, dt, T, H, eps, dz, dw, ws, n, None)

    assert f(T=-1) == INVALID and f(H=0) == INVALID and f(dt=FP8) == INVALID and f(eps=0.0) == INVALID
    assert f(H=100) == UNSUPPORTED and f(H=16392) == UNSUPPORTED
    for name in ("dy", "z", "w", "dz", "dw"):
        assert f(**{name: None}) == INVALID
    for name in ("dy", "z", "w", "d", "dz", "ws"):
        assert f(**{name: ODD}) == INVALID
    for name, value in (("dz", B), ("dz", D), ("dz", F), ("dz", G), ("dw", A), ("dw", B), ("dw", G), ("ws", A), ("ws", D)):
        assert f(**{name: value}) == INVALID and "same buffer" in binding.last_error()
    assert f(ws=None) == WORKSPACE
    need = L.moe_rmsnorm_backward_workspace_size(4, 256)
    assert need > 0 and f(n=need - 1) == WORKSPACE
    assert f(T=0, dw=None) == INVALID
    size = L.moe_rmsnorm_backward_workspace_size
    assert size(0, 256) == 0 and size(-1, 256) == 0 and size(4, 100) == 0
    assert size(1 << 30, 16384) == size(1 << 20, 16384)     # bounded: not a row for each token


def test_dispatch_validation(L):
    def f(x=A, xs=None, dt=BF16, T=4, H=256, k=2, sh=0, up=B, rows=D, rs=None):
        return L.moe_dispatch(x, xs, dt, T, H, k, sh, up, rows, rs, None)

    assert f(T=-1) == INVALID and f(k=0) == INVALID and f(sh=-1) == INVALID and f(sh=65) == INVALID
    assert f(k=9) == UNSUPPORTED and f(H=100) == UNSUPPORTED and f(dt=5) == INVALID and f(H=0) == INVALID
    assert f(dt=FP8, H=264, xs=E, rs=F) == UNSUPPORTED
    assert f(dt=FP8) == INVALID and f(dt=FP8, xs=E) == INVALID and f(xs=E, rs=F) == INVALID
    assert f(rows=A) == INVALID and f(rows=B) == INVALID and f(dt=FP8, xs=E, rs=E) == INVALID
    assert f(dt=FP8, xs=E, rs=A) == INVALID and f(dt=FP8, xs=E, rs=D) == INVALID
    assert f(x=None) == INVALID and f(up=None) == INVALID and f(rows=None) == INVALID
    assert f(x=ODD) == INVALID and f(rows=ODD) == INVALID
    assert f(T=1 << 29, k=4) == UNSUPPORTED and f(H=(1 << 28) + 8) == UNSUPPORTED
    assert f(T=0, x=None, up=None, rows=None) == OK

    def g(d=A, dt=BF16, up=B, T=4, k=2, H=256, sh=0, dx=D, dxt=BF16):
        return L.moe_dispatch_backward(d, dt, up, T, k, H, sh, dx, dxt, None)

    assert g(dt=FP8) == INVALID and g(dxt=FP8) == INVALID and g(k=9) == UNSUPPORTED and g(H=4) == UNSUPPORTED
    assert g(d=None) == INVALID and g(up=None) == INVALID and g(dx=None) == INVALID
    assert g(d=ODD) == INVALID and g(dx=ODD) == INVALID and g(dx=A) == INVALID
    assert g(T=0, d=None, up=None, dx=None) == OK


def test_finalize_backward_validation(L):
    def f(dy=A, dyt=BF16, r=B, dt=BF16, up=D, sc=E, T=4, k=2, H=256, sh=0, d=F, ds=G):
        return L.moe_finalize_backward(dy, dyt, r, dt, up, sc, T, k, H, sh, d, ds, None)

    assert f(T=-1) == INVALID and f(dyt=FP8) == INVALID and f(dt=FP8) == INVALID
    assert f(k=9) == UNSUPPORTED and f(H=12) == UNSUPPORTED and f(T=1 << 29, k=4) == UNSUPPORTED
    for name in ("dy", "r", "up", "sc", "d", "ds"):
        assert f(**{name: None}) == INVALID
    for name in ("dy", "r", "d"):
        assert f(**{name: ODD}) == INVALID
    for name, value in (("d", A), ("d", E), ("ds", A), ("ds", B), ("ds", E), ("ds", F)):
        assert f(**{name: value}) == INVALID and "same buffer" in binding.last_error()
    assert f(T=0, dy=None, r=None, up=None, sc=None, d=None, ds=None) == OK


def test_route_backward_validation(L):
    def f(l=A, i=B, d=D, T=4, E=16, method=0, k=2, sc=1.0, flags=0, out=F):
        return L.moe_route_backward(l, i, d, T, E, method, k, sc, flags, out, None)

    assert f(T=-1) == INVALID and f(k=0) == INVALID and f(k=17) == INVALID and f(E=0) == INVALID
    assert f(E=300) == UNSUPPORTED and f(E=64, k=9) == UNSUPPORTED
    assert f(method=7) == UNSUPPORTED and f(method=8) == UNSUPPORTED
    assert f(method=9) == INVALID and f(method=-1) == INVALID and f(flags=2) == INVALID
    assert f(sc=float("nan")) == INVALID
    for name in ("l", "i", "d", "out"):
        assert f(**{name: None}) == INVALID
    assert f(out=ODD) == INVALID and f(out=A) == INVALID and f(out=D) == INVALID
    assert f(T=0, l=None, i=None, d=None, out=None) == OK


def test_swiglu_validation(L):
    def f(gu=A, dt=BF16, rows=4, I=256, h=B, hq=None, hs=None, q=None, qs=None):
        return L.moe_swiglu(gu, dt, rows, I, h, hq, hs, q, qs, None)

    assert f(rows=-1) == INVALID and f(I=0) == INVALID and f(dt=FP8) == INVALID and f(gu=None) == INVALID
    assert f(I=12) == UNSUPPORTED and f(I=264, q=F, qs=G) == UNSUPPORTED and f(I=264, hq=D, hs=E) == UNSUPPORTED
    assert f(rows=(1 << 30) + 1) == UNSUPPORTED and f(I=(1 << 29) + 128) == UNSUPPORTED
    assert f(h=None) == INVALID
    assert f(hq=D) == INVALID and f(hs=E) == INVALID and f(q=F) == INVALID and f(qs=G) == INVALID
    assert f(gu=ODD) == INVALID and f(h=ODD) == INVALID
    assert f(hq=ODD, hs=E) == INVALID and f(q=ODD, qs=G) == INVALID
    full = dict(gu=A, h=B, hq=D, hs=E, q=F, qs=G)
    for a in full:
        for b in full:
            if a != b:
                assert f(**{**full, a: full[b]}) == INVALID and "same buffer" in binding.last_error()
    assert f(rows=0, gu=None, h=None) == OK

    def g(dh=A, dt=BF16, q=B, qs=D, rows=4, I=256, d=E, h=None):
        return L.moe_swiglu_backward(dh, dt, q, qs, rows, I, d, h, None)

    assert g(rows=-1) == INVALID and g(I=0) == INVALID and g(dt=FP8) == INVALID
    assert g(I=264) == UNSUPPORTED
    for name in ("dh", "q", "qs", "d"):
        assert g(**{name: None}) == INVALID
    for name in ("dh", "q", "d", "h"):
        assert g(**{name: ODD}) == INVALID
    for name, value in (("d", A), ("d", B), ("d", D), ("h", B), ("h", E)):
        assert g(**{name: value}) == INVALID and "same buffer" in binding.last_error()
    assert g(rows=0, dh=None, q=None, qs=None, d=None) == OK


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 256), torch.ones(256)
    i = torch.zeros(8, dtype=torch.int32)
    calls = [lambda: moe.rmsnorm(x, w), lambda: moe.rmsnorm_backward(x, x, w),
             lambda: moe.dispatch(x, i, 2), lambda: moe.dispatch_backward(x, i, 2),
             lambda: moe.finalize_backward(x, x, i, torch.zeros(4, 2)),
             lambda: moe.route_backward(x, i.view(4, 2), torch.zeros(4, 2), 0),
             lambda: moe.swiglu(x), lambda: moe.swiglu_backward(x, x, x)]
    for call in calls:
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call()


# ----------------------------------------------------- the binding's native half
def test_call_checks_its_arguments(L):
    """Wrong counts, numbers that do not fit and buffers that are none are refused before the
    device is touched."""
    a = (None, 1, None, None, 1, 1, 8, 0, None, 0)
    for args, error in ((a[:-1], TypeError), (a + (0,), TypeError), ((3,) + a[1:], TypeError),
                        (a[:4] + (2 ** 31,) + a[5:], OverflowError), (a[:4] + (1.5,) + a[5:], TypeError),
                        ((torch.zeros(8),) + a[1:], ValueError)):
        with pytest.raises(error):
            binding._call("moe_finalize", "cuda:0", *args)
    with pytest.raises(AttributeError, match="no entry point moe_nothing"):
        binding._call("moe_nothing", "cuda:0")
    with pytest.raises(TypeError):
        binding._marshal.call("moe_finalize", "cuda:0", *a)  # a torch.device


def test_call_covers_every_kernel_entry():
    """Each entry point that launches is known to the native half (it asks for its arguments)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moe.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    launching = re.findall(r"moe_status (moe_\w+)\([^;]*void\* stream\);", text)
    assert len(launching) >= 17
    for fn in launching:
        with pytest.raises(TypeError, match=fn):
            binding._call(fn, "cuda:0")


def test_check_accepts_and_refuses():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        binding._dev(x, "x", torch.float32, (4, 8))
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        binding._dev(x, "x", shape=(4, 8))
    with pytest.raises(AttributeError):
        binding._dev(None, "x", torch.float32)
    for call in (lambda: binding._dev(), lambda: binding._dev(x), lambda: binding._dev(x, "x", type=3),
                 lambda: binding._dev(x, "x", None, None, None)):
        with pytest.raises(TypeError):
            call()
