"""The layer for few tokens without a GPU: the host checks (the pointers here are never dereferenced)."""
import ctypes as C
import os

import pytest
import torch

import mixture_experts_layer_07_amd as moe
from mixture_experts_layer_07_amd import binding

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
ODD = C.c_void_p((1 << 20) + 4)
A, B, D, E, F, G, I, J, K, M, N = (C.c_void_p(n << 24) for n in range(1, 12))
F32, BF16, FP8, MX = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from mixture_experts_layer_07_amd import build
        build.build(verbose=False)
    return moe.lib()


def test_validation(L):
    def f(x=A, act=BF16, lg=B, T=4, H=256, I_=128, E_=8, method=1, k=2, ng=1, tg=1, bias=None, sc=1.0, flags=0, sh=0,
          w13=D, w2=E, wdt=BF16, s13=None, s2=None, ids=F, scales=G, y=I, ws=J, n=1 << 30):
        return L.moe_layer_few(x, act, lg, T, H, I_, E_, method, k, ng, tg, bias, sc, flags, sh, w13, w2, wdt, s13, s2,
                               ids, scales, y, ws, n, None)

    assert f(T=-1) == INVALID and f(k=0) == INVALID and f(k=9) == INVALID and f(sh=65) == INVALID and f(E_=0) == INVALID
    assert f(T=33) == UNSUPPORTED and "32 tokens" in binding.last_error()
    assert f(E_=300) == UNSUPPORTED and f(E_=64, k=9) == UNSUPPORTED
    assert f(H=0) == INVALID and f(I_=-128) == INVALID and f(H=192) == UNSUPPORTED and f(I_=64) == UNSUPPORTED
    assert f(H=(1 << 20) + 128) == UNSUPPORTED
    # one expert's w13 and h have to be under 4 GiB (T = 0: nothing else is looked at)
    big, n = 1 << 20, 1 << 40
    for wdt, rows in ((F32, 512), (BF16, 1024), (FP8, 2048), (MX, 4096)):
        how = dict(act=F32 if wdt == F32 else BF16, wdt=wdt, T=0, H=big)
        assert f(**how, I_=rows) == UNSUPPORTED and "w13" in binding.last_error(), wdt
        assert f(**how, I_=rows - 128) == OK, wdt
    assert f(T=32, k=8, E_=64, sh=56, H=128, I_=big, n=n) == UNSUPPORTED and "h of 2048 rows" in binding.last_error()
    assert L.moe_layer_few_workspace_size(32, 128, big, 64, 8, 56, BF16) == 0
    assert L.moe_layer_few_workspace_size(32, 128, big - 128, 64, 8, 56, BF16) > (1 << 32) - (1 << 20)
    assert f(act=FP8) == INVALID and f(act=MX) == INVALID and f(wdt=4) == INVALID and f(wdt=-1) == INVALID
    assert f(act=F32) == UNSUPPORTED and f(wdt=F32) == UNSUPPORTED and f(act=F32, wdt=MX) == UNSUPPORTED
    # the routing's own refusals
    assert f(method=7) == UNSUPPORTED and f(method=9) == INVALID and f(flags=2) == INVALID and f(sc=float("nan")) == INVALID
    assert f(method=2, ng=3) == INVALID and f(method=2, ng=8) == INVALID and f(method=2, ng=2, tg=3) == INVALID
    for name in ("x", "lg", "w13", "w2", "ids", "scales", "y"):
        assert f(**{name: None}) == INVALID, name
    for wdt in (FP8, MX):
        assert f(wdt=wdt) == INVALID and f(wdt=wdt, s13=K) == INVALID and f(wdt=wdt, s2=K) == INVALID
    full = dict(x=A, lg=B, w13=D, w2=E, wdt=MX, s13=K, s2=M, method=2, bias=N)
    for name in ("x", "w13", "w2", "s13", "s2", "y", "ws"):
        assert f(**{**full, name: ODD}) == INVALID and "aligned" in binding.last_error(), name
    buffers = dict(x=A, lg=B, w13=D, w2=E, s13=K, s2=M, bias=N, ids=F, scales=G, y=I, ws=J)
    for out in ("ids", "scales", "y", "ws"):
        for other, value in buffers.items():
            if other != out:
                assert f(**{**full, out: value}) == INVALID and "same buffer" in binding.last_error(), (out, other)
    assert f(ws=None) == WORKSPACE
    size = L.moe_layer_few_workspace_size
    need = size(4, 256, 128, 8, 2, 0, BF16)
    assert f(n=need - 1) == WORKSPACE
    assert need >= 4 * 2 * 128 * 2 and size(4, 256, 128, 8, 2, 1, F32) >= 4 * 3 * 128 * 4  # h and what goes with it
    assert size(0, 256, 128, 8, 2, 0, BF16) == 0 and size(33, 256, 128, 8, 2, 0, BF16) == 0
    assert size(4, 256, 100, 8, 2, 0, BF16) == 0 and size(4, 256, 128, 8, 2, 0, FP8) == 0
    assert f(T=0, x=None, ws=None) == OK


def test_binding_refuses_host_tensors():
    x, l, w = torch.zeros(4, 128), torch.zeros(4, 8), torch.zeros(8, 256, 128)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        moe.layer_few(x, l, w, w, 2, 0)
