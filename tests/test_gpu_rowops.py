"""The row operators on the GPU against their 64-bit forms.

Tolerances are sums of what the arithmetic may lose: half a step of the output's
type for its one rounding, and for the fp32 work before it a number of fp32
half-steps (2^-24) times the size of the terms that were added (the references
return that size).  Where no rounding but the output's own is made, results
are compared bit for bit.  Outputs lie in poisoned buffers whose surroundings
must stay as they were.
"""
import numpy as np
import pytest
import torch

import oracle
import mixture_experts_layer_07_amd as moe
import rowops_ref as ref
from mixture_experts_layer_07_amd import binding
from rowops_ref import EPS32, F64, half_step

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, FP, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = [BF, FP]
GUARD = 256


def rnd(*shape, seed=0, scale=1.0, dt=FP):
    v = np.random.default_rng([seed, *shape]).standard_normal(shape, dtype=np.float32) * np.float32(scale)
    return torch.from_numpy(v).to(dt)


def outliers(*shape, seed=0, dt=FP):
    """Hidden states: normal, a few channels 12 times as large, rows of different sizes."""
    v = rnd(*shape, seed=seed)
    v[:, ::97] *= 12
    v *= torch.logspace(-2, 2, shape[0])[:, None]
    return v.to(dt)


class Guarded:
    """Outputs inside poisoned buffers."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dt):
        n = int(np.prod(shape)) * torch.empty((), dtype=dt).element_size()
        buf = torch.full((GUARD + n + GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
        self.all.append((buf, n))
        return buf[GUARD:GUARD + n].view(dt).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            assert bool((buf[:GUARD] == 0xA5).all()) and bool((buf[GUARD + n:] == 0xA5).all()), "written outside"


def within(got, want, tol, what):
    got, want, tol = got.detach().cpu().to(F64), want.to(F64), tol.to(F64)
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst by "
                                 f"{float(((got - want).abs() / tol.clamp_min(1e-300))[bad].max()):.3g} tolerances")


def bits(a):
    return a.detach().cpu().contiguous().view(torch.uint8)


def same(a, b, what):
    assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(bits(a), bits(b)), what


def codes_close(q, s, v, rel, what):
    """Codes q and scales s of 1x128 blocks of v, computed in fp32 with relative error rel."""
    rows, cols = v.shape
    amax = v.abs().view(rows, cols // 128, 128).amax(2)
    within(s, amax / 448, amax / 448 * (rel + 2 * EPS32), what + " scales")
    # rel moves the value (and the block's scale) before the rounding: a code next to a border
    # may fall on its other side, which costs half a step either way and what moved it
    s = s.cpu()
    within(ref.values(q.cpu(), s), v, ref.code_tolerance(v, s) * (1 + 2 ** -10) + v.abs() * 4 * (rel + EPS32),
           what + " codes")


def spread(T, E, k, seed=0):
    """Places of a skewed routing (most experts of a small batch empty), by the library's oracle."""
    rng = np.random.default_rng([seed, T, E, k])
    logits = rng.standard_normal((T, E)) - 1.2 * np.log(rng.permutation(E) + 1.0)
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32)
    _, _, up = oracle.permute(np.ascontiguousarray(ids), E, 0)
    return torch.from_numpy(up)


# ----------------------------------------------------------------------- norm
# the fp32 sum of H squares goes in chains of at most 32 (a thread's) and 9 (lanes, waves) additions;
# half of its relative error reaches c, then the square root's inverse (2) and two products
NORM = 48 * EPS32

NORM_SHAPES = [(1, 8), (3, 248), (5, 256), (63, 512), (33, 520), (7, 2048), (4, 2056), (9, 4096), (5, 7168),
               (2, 8192), (3, 8200), (2, 16384), (4100, 128)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(T, H, residual, dt):
    x, w = outliers(T, H, dt=dt), (1 + 0.1 * rnd(H, seed=1)).to(dt)
    r = outliers(T, H, seed=2, dt=dt) if residual else None
    q = H % 128 == 0
    g = Guarded()
    out = (g((T, H), dt), g((T, H), dt) if residual else None, g((T, H), F8) if q else None,
           g((T, H // 128), FP) if q else None)
    y, total, yq, ys = moe.rmsnorm(x.to(DEV), w.to(DEV), 1e-5, residual=None if r is None else r.to(DEV),
                                   quantize=q, out=out)
    g.check()
    z = x
    if residual:
        z = (x.float() + r.float()).to(dt)
        same(total.cpu(), z, "total")
    want = ref.rmsnorm(z, w, float(np.float32(1e-5)))
    within(y, want, want.abs() * (half_step(dt) + NORM * 1.01) + 2.0 ** -126, "y")
    if q:
        codes_close(yq, ys, want, NORM, "y")
        if dt == FP:  # the codes are those of the fp32 y
            q2, s2 = moe.quantize_fp8(y)
            same(yq, q2, "codes of y")
            same(ys, s2, "scales of y")
        only = moe.rmsnorm(x.to(DEV), w.to(DEV), 1e-5, residual=None if r is None else r.to(DEV), quantize=True,
                           want_y=False)
        assert only[0] is None
        same(only[2], yq, "codes without y")
        same(only[3], ys, "scales without y")


@pytest.mark.parametrize("dt", TYPES)
def test_rmsnorm_in_place(dt):
    T, H = 37, 1024
    x, r, w = outliers(T, H, dt=dt).to(DEV), rnd(T, H, seed=2, dt=dt).to(DEV), rnd(H, seed=1, dt=dt).to(DEV)
    y, total, yq, ys = moe.rmsnorm(x, w, residual=r, quantize=True)
    for into in ("x", "residual"):
        a, b = x.clone(), r.clone()
        t2 = a if into == "x" else b
        got = moe.rmsnorm(a, w, residual=b, quantize=True, out=(None, t2, None, None))
        assert got[1].data_ptr() == t2.data_ptr()
        for m, n, what in zip(got, (y, total, yq, ys), ("y", "total", "codes", "scales")):
            same(m, n, f"{what} with total in {into}")
    a = x.clone()
    got = moe.rmsnorm(a, w, out=(a, None, None, None))[0]
    same(got, moe.rmsnorm(x, w)[0], "y in x")


@pytest.mark.parametrize("dt", TYPES)
def test_rmsnorm_special_rows(dt):
    """Zero rows, subnormal and huge values, a NaN row and an infinite one beside ordinary ones."""
    T, H = 12, 512
    x, w = rnd(T, H, dt=dt), torch.ones(H, dtype=dt)
    x[1] = 0
    x[2] = -0.0
    x[3] = 1e-30
    x[4] *= 1e15
    x[5, 7] = float("nan")
    x[6, 500] = float("inf")
    x[8, :256] = 0
    got = [None if t is None else t.cpu() for t in moe.rmsnorm(x.to(DEV), w.to(DEV), 1e-6, quantize=True)]
    fine = [i for i in range(T) if i not in (5, 6)]
    want = ref.rmsnorm(x[fine], w, float(np.float32(1e-6)))
    within(got[0][fine], want, want.abs() * (half_step(dt) + NORM * 1.01) + 2.0 ** -126, "y")
    codes_close(got[2][fine], got[3][fine], want, NORM, "y")
    assert bool((got[2].view(torch.uint8)[1] & 0x7F == 0).all()) and bool((got[3][1] == 0).all())
    assert bool((got[3][8, :2] == 0).all()) and bool((got[3][8, 2:] > 0).all())
    assert bool(got[0][5].isnan().all())
    # the others are what they are without the bad rows
    alone = moe.rmsnorm(x[fine].contiguous().to(DEV), w.to(DEV), 1e-6, quantize=True)
    same(got[0][fine], alone[0].cpu(), "rows beside NaN")
    same(got[2][fine], alone[2].cpu(), "codes beside NaN")


def dweight_depth(T, H):
    """Additions in the longest chain of dweight: a partial sum's rows (spread over up to 512 sums, or
    all of 4 where one workgroup takes them), its waves (4, or 16 that then are all), the 16 partial
    sums of a run, 32 runs."""
    return -(-T // 512) + 4 + 16 + 32


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H", NORM_SHAPES + [(2500, 520), (1300, 2056)])
@pytest.mark.parametrize("dsum", [False, True])
def test_rmsnorm_backward(T, H, dsum, dt):
    z, w = outliers(T, H, dt=dt), (1 + 0.1 * rnd(H, seed=1)).to(dt)
    dy = rnd(T, H, seed=3, scale=1e-2, dt=dt)
    d = rnd(T, H, seed=4, scale=1e-2, dt=dt) if dsum else None
    g = Guarded()
    ws = g((max(1, int(moe.lib().moe_rmsnorm_backward_workspace_size(T, H))),), torch.uint8)
    out = (g((T, H), dt), g((H,), FP))
    args = (dy.to(DEV), z.to(DEV), w.to(DEV), 1e-5)
    dd = None if d is None else d.to(DEV)
    dz, dw = moe.rmsnorm_backward(*args, dsum=dd, ws=ws, out=out)
    g.check()
    want, wantw, size, sizew = ref.rmsnorm_backward(dy, z, w, float(np.float32(1e-5)), d)
    within(dz, want, want.abs() * half_step(dt) + size * (3 * NORM + 8 * EPS32) * 1.01, "dz")
    within(dw, wantw, sizew * ((dweight_depth(T, H) + 2) * EPS32 + NORM), "dweight")
    dz2, dw2 = moe.rmsnorm_backward(*args, dsum=dd)
    same(dz, dz2, "dz again")
    same(dw, dw2, "dweight again")
    for into, src in ((0, dy), (1, d)):  # dz over dy, over dsum
        if src is None:
            continue
        a = [dy.to(DEV), dd]
        a[into] = src.to(DEV).clone()
        dz3, dw3 = moe.rmsnorm_backward(a[0], args[1], args[2], 1e-5, dsum=a[1], out=(a[into], None))
        same(dz, dz3, "dz in place")
        same(dw, dw3, "dweight in place")


def test_rmsnorm_backward_against_differences():
    T, H = 6, 256
    z, w, dy = rnd(T, H), 1 + 0.1 * rnd(H, seed=1), rnd(T, H, seed=2)
    dz, dw = moe.rmsnorm_backward(dy.to(DEV), z.to(DEV), w.to(DEV), 1e-5)
    e = float(np.float32(1e-5))
    for seed in range(4):
        v, u = rnd(T, H, seed=10 + seed).to(F64), rnd(H, seed=20 + seed).to(F64)
        a = ref.differences(lambda x: (ref.rmsnorm(x, w, e) * dy.to(F64)).sum(), z.to(F64), v, 1e-5)
        b = ref.differences(lambda x: (ref.rmsnorm(z, x, e) * dy.to(F64)).sum(), w.to(F64), u, 1e-5)
        # sums of T*H terms of order 1, each off by some 2^-18
        assert abs(float((dz.cpu().to(F64) * v).sum()) - a) < 1e-2
        assert abs(float((dw.cpu().to(F64) * u).sum()) - b) < 1e-2


def test_rmsnorm_backward_tiny_eps():
    """A zero row under a tiny eps: c is large, its third power would overflow."""
    T, H = 5, 256
    z, w, dy = rnd(T, H), torch.ones(H), rnd(T, H, seed=2)
    z[2] = 0
    dz, dw = moe.rmsnorm_backward(dy.to(DEV), z.to(DEV), w.to(DEV), 1e-30)
    want, wantw, size, sizew = ref.rmsnorm_backward(dy, z, w, float(np.float32(1e-30)))
    within(dz, want, want.abs() * half_step(FP) + size * (3 * NORM + 8 * EPS32) * 1.01, "dz")
    within(dw, wantw, sizew * ((dweight_depth(T, H) + 2) * EPS32 + NORM), "dweight")


def test_rmsnorm_backward_of_no_rows():
    w = torch.ones(264, device=DEV)
    e = torch.empty(0, 264, device=DEV)
    dw = torch.full((264,), 7.0, device=DEV)
    dz, got = moe.rmsnorm_backward(e, e, w, out=(None, dw))
    assert dz.shape == (0, 264) and got is dw and bool((dw == 0).all())


# ------------------------------------------------------- rows in expert order
PLACES = [(1, 8, 8, 1, 0), (1, 264, 1, 1, 0), (3, 128, 4, 2, 2), (65, 1024, 8, 2, 0), (37, 7168, 256, 8, 1),
          (129, 520, 16, 3, 1), (20, 16384, 12, 6, 0), (1100, 256, 64, 8, 3), (5, 2048, 8, 8, 64)]


@pytest.mark.parametrize("dt", [BF, FP, F8])
@pytest.mark.parametrize("T,H,E,k,sh", PLACES)
def test_dispatch(T, H, E, k, sh, dt):
    if dt == F8 and H % 128:
        H = 128 * (1 + H // 128)
    up = spread(T, E, k)
    R = T * (k + sh)
    x = rnd(T, H, dt=FP if dt == F8 else dt)
    g = Guarded()
    if dt == F8:
        x, s = x.to(F8), rnd(T, H // 128, seed=1)
        rows, rs = moe.dispatch(x.to(DEV), up.to(DEV), k, sh, x_scale=s.to(DEV),
                                out=(g((R, H), F8), g((R, H // 128), FP)))
        same(rs.cpu(), ref.dispatch(s, up, k, sh), "scales")
        same(rows.cpu(), ref.dispatch(x.view(torch.uint8), up, k, sh).view(F8), "rows")
    else:
        rows = moe.dispatch(x.to(DEV), up.to(DEV), k, sh, out=g((R, H), dt))
        same(rows.cpu(), ref.dispatch(x, up, k, sh), "rows")
    g.check()


@pytest.mark.parametrize("dt,dxt", [(BF, BF), (FP, FP), (BF, FP), (FP, BF)])
@pytest.mark.parametrize("T,H,E,k,sh", PLACES)
def test_dispatch_backward(T, H, E, k, sh, dt, dxt):
    up = spread(T, E, k)
    d = rnd(T * (k + sh), H, seed=5, dt=dt)
    g = Guarded()
    dx = moe.dispatch_backward(d.to(DEV), up.to(DEV), k, sh, out_dtype=dxt, out=g((T, H), dxt))
    g.check()
    want, size = ref.dispatch_backward(d, up, k, sh)
    within(dx, want, want.abs() * half_step(dxt) + size * (k + sh + 1) * EPS32, "dx")
    # moe_finalize with every scale 1 adds in the same order
    if dxt == dt:
        same(dx, moe.finalize(d.to(DEV), up.to(DEV), torch.ones(T, k, device=DEV), sh), "finalize of ones")


@pytest.mark.parametrize("dyt,dt", [(BF, BF), (FP, FP), (BF, FP), (FP, BF)])
@pytest.mark.parametrize("T,H,E,k,sh", PLACES)
def test_finalize_backward(T, H, E, k, sh, dyt, dt):
    up = spread(T, E, k)
    R = T * (k + sh)
    fc2, dy, sc = rnd(R, H, seed=6, dt=dt), rnd(T, H, seed=7, scale=1e-2, dt=dyt), rnd(T, k, seed=8)
    g = Guarded()
    d, ds = moe.finalize_backward(dy.to(DEV), fc2.to(DEV), up.to(DEV), sc.to(DEV), sh,
                                  out=(g((R, H), dt), g((T, k), FP)))
    g.check()
    # one fp32 product and its rounding
    want = torch.zeros(R, H, dtype=dt)
    want[up.long()] = (sc.reshape(-1, 1) * dy.float().repeat_interleave(k, 0)).to(dt)
    if sh:
        want[T * k:] = dy.float().repeat(sh, 1).to(dt)
    same(d.cpu(), want, "d_fc2")
    terms = dy.to(F64)[:, None] * fc2.to(F64)[up.long()].view(T, k, H)
    chain = 8 * -(-H // 2048) + 12  # a thread's products, then lanes and waves
    within(ds, terms.sum(2), terms.abs().sum(2) * chain * EPS32, "d_scales")
    a = fc2.to(DEV).clone()
    d2, ds2 = moe.finalize_backward(dy.to(DEV), a, up.to(DEV), sc.to(DEV), sh, out=(a, None))
    same(d2, d, "in place")
    same(ds2, ds, "d_scales in place")


@pytest.mark.parametrize("dt", TYPES)
def test_dropped_pairs(dt):
    """Entries outside [0, T*k) are dropped pairs: nothing is written or added for them."""
    T, H, E, k, sh = 40, 512, 8, 3, 1
    up = spread(T, E, k)
    drop = torch.from_numpy(np.random.default_rng(3).random(T * k) < 0.3)
    up[drop] = torch.tensor([-1, T * k, 2 ** 31 - 1, -2 ** 31])[torch.arange(int(drop.sum())) % 4].int()
    up[:k] = -1  # a token without any
    named = torch.zeros(T * (k + sh), dtype=torch.bool)
    named[up[(up >= 0) & (up < T * k)].long()] = True
    named[T * k:] = True
    x = rnd(T, H, dt=dt)
    rows = torch.full((T * (k + sh), H), 3.0, dtype=dt, device=DEV)
    moe.dispatch(x.to(DEV), up.to(DEV), k, sh, out=rows)
    assert bool((rows.cpu()[~named] == 3).all())
    for t in range(T):
        for r in [int(v) for v in up[t * k:(t + 1) * k] if 0 <= v < T * k] + [T * k + t]:
            assert torch.equal(rows.cpu()[r], x[t])
    d = rnd(T * (k + sh), H, seed=1, dt=dt)
    d[~named] = float("nan")  # never read
    dx = moe.dispatch_backward(d.to(DEV), up.to(DEV), k, sh)
    want, size = ref.dispatch_backward(d, up, k, sh)
    within(dx, want, want.abs() * half_step(dt) + size * (k + sh) * EPS32, "dx")
    sc, dy = rnd(T, k, seed=2), rnd(T, H, seed=4, dt=dt)
    out = torch.full((T * (k + sh), H), 3.0, dtype=dt, device=DEV)
    _, ds = moe.finalize_backward(dy.to(DEV), d.to(DEV), up.to(DEV), sc.to(DEV), sh, out=(out, None))
    assert bool((out.cpu()[~named] == 3).all())
    kept = ((up >= 0) & (up < T * k)).view(T, k)
    assert bool((ds.cpu()[~kept] == 0).all()) and not bool(ds.isnan().any())


# -------------------------------------------------------------- routing weights
ROUTES = [(1, 1, 1), (11, 2, 2), (1, 8, 1), (1, 256, 8), (31, 7, 7), (33, 65, 3), (100, 256, 8), (64, 12, 2), (1029, 9, 4), (70, 255, 5)]


@pytest.mark.parametrize("method,renorm", [(0, False), (0, True), (1, False), (2, False), (3, False), (4, False),
                                           (5, False), (6, False)])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route_backward(T, E, k, method, renorm):
    l, ds = rnd(T, E, scale=2.0), rnd(T, k, seed=1)
    ids = (l + 0.3 * rnd(T, E, seed=2)).topk(k, 1).indices.int()
    g = Guarded()
    got = moe.route_backward(l.to(DEV), ids.to(DEV), ds.to(DEV), method, 2.5, renorm, out=g((T, E), FP))
    g.check()
    want, size = ref.route_backward(l, ids, ds, method, 2.5, renorm)
    # fp64 and one rounding; plain softmax takes exponentials of fp32 differences (up to 16 here)
    within(got, want, size * ((24 if method == 0 and not renorm else 1.5) * EPS32) + 2.0 ** -140, "d_logits")
    if k == 1 and (renorm or method in (1, 4, 5, 6)):
        assert bool((got == 0).all())


@pytest.mark.parametrize("method", range(7))
def test_route_backward_of_the_routing(method):
    """From moe_route's own ids; and the slope of its scales along a direction."""
    T, E, k = 50, 64, 6
    l, ds, v = rnd(T, E), rnd(T, k, seed=1), rnd(T, E, seed=2).to(F64)
    bias = 0.1 * rnd(E, seed=3)
    group = (8, 4) if method == 2 else (1, 1)
    ids, _ = moe.route(l.to(DEV), k, method, *group, bias.to(DEV) if method in (2, 5) else None, 2.5)
    got = moe.route_backward(l.to(DEV), ids, ds.to(DEV), method, 2.5).cpu()
    want = ref.differences(lambda a: (ref.route_scales(a, ids.cpu(), method, 2.5, False) * ds.to(F64)).sum(),
                           l.to(F64), v, 1e-5)
    assert abs(float((got.to(F64) * v).sum()) - want) < 1e-4  # hundreds of terms below 1, 2^-22 each


@pytest.mark.parametrize("method", range(7))
def test_route_backward_special_rows(method):
    T, E, k = 9, 40, 4
    l, ds = rnd(T, E), rnd(T, k, seed=1)
    ids = torch.arange(T * k).view(T, k).int() % E
    l[0] = float("-inf")                      # a mask that leaves nothing
    l[1, ids[1, 1:].long()] = float("-inf")   # one kept expert left
    l[2] = torch.finfo(FP).min                # masks of the type's lowest value
    l[3] = -90.0                              # sigmoids far below fp32's exponentials
    l[4] = 60.0
    l[5, 3] = float("nan")
    l[6] = 300 * l[6].sign()
    ids[7, 2] = -1                            # dropped pairs
    ids[7, 3] = E
    got = moe.route_backward(l.to(DEV), ids.to(DEV), ds.to(DEV), method, 1.0).cpu()
    assert bool((got[0] == 0).all())
    rows = [1, 3, 4, 6, 8] + ([2] if method in (0, 1, 4) else [])
    want, size = ref.route_backward(l[rows], ids[rows], ds[rows], method, 1.0, False)
    within(got[rows], want, size * (24 + (600 if method == 0 else 0)) * EPS32 + 2.0 ** -126, "d_logits")
    assert not bool(got[2].isnan().any())
    # a dropped pair takes no part: the same as a shorter list
    want, size = ref.route_backward(l[7:8], ids[7:8, :2], ds[7:8, :2], method, 1.0, False)
    within(got[7:8], want, size * 24 * EPS32 + 2.0 ** -126, "with dropped pairs")


@pytest.mark.parametrize("method", range(7))
def test_route_backward_expert_twice(method):
    T, E, k = 40, 16, 5
    l, ds = rnd(T, E), rnd(T, k, seed=1)
    ids = torch.from_numpy(np.random.default_rng(0).integers(0, E, (T, k))).int()
    ids[0] = 3
    a = moe.route_backward(l.to(DEV), ids.to(DEV), ds.to(DEV), method, 1.0)
    want, size = ref.route_backward(l, ids, ds, method, 1.0, False)
    within(a, want, size * 24 * EPS32 + 2.0 ** -126, "d_logits")
    same(a, moe.route_backward(l.to(DEV), ids.to(DEV), ds.to(DEV), method, 1.0), "again")


# ------------------------------------------------------------------ activation
SWIGLU = [(1, 8), (3, 24), (5, 128), (17, 256), (9, 1408), (3, 2048), (2, 14336), (1, 16384), (700, 384), (33, 640)]


def silu_rel(g):
    """e^-g by the product form: relative error up to 2^-23 |g| + a few steps; the rest 8 steps."""
    return (2 * g.abs() + 12) * EPS32


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,I", SWIGLU)
def test_swiglu(rows, I, dt):
    gu = outliers(rows, 2 * I, dt=dt)
    q = I % 128 == 0
    g = Guarded()
    out = (g((rows, I), dt), g((rows, I), F8) if q else None, g((rows, I // 128), FP) if q else None,
           g((rows, 2 * I), F8) if q else None, g((rows, 2 * I // 128), FP) if q else None)
    h, hq, hs, gq, gs = moe.swiglu(gu.to(DEV), quantize=q, checkpoint=q, want_h=True, out=out)
    g.check()
    want = ref.swiglu(gu)
    gate, up = gu[:, :I].to(F64), gu[:, I:].to(F64)
    floor = (gate * up).abs() * 2.0 ** -125 + 2.0 ** -126  # sigmoids below fp32's normal values
    within(h, want, want.abs() * (half_step(dt) + 1.01 * silu_rel(gate)) + floor, "h")
    if not q:
        return
    cq, cs = oracle.quantize_fp8(gu if dt == FP else gu.view(torch.int16).numpy(), "f32" if dt == FP else "bf16")
    assert np.array_equal(bits(gq).numpy().reshape(cq.shape), cq), "checkpoint codes"
    assert np.array_equal(gs.cpu().numpy(), cs), "checkpoint scales"
    q2, s2 = moe.quantize_fp8(gu.to(DEV))
    same(gq, q2, "checkpoint of the quantiser")
    same(gs, s2, "scales of the quantiser")
    # gates of the block's largest h are below 2^10 here
    codes_close(hq, hs, want, 2060 * EPS32, "h")
    if dt == FP:
        q3, s3 = moe.quantize_fp8(h)
        same(hq, q3, "codes of h")
        same(hs, s3, "scales of h")
    only = moe.swiglu(gu.to(DEV), quantize=True)
    assert only[0] is None and only[3] is None
    same(only[1], hq, "codes alone")
    same(only[2], hs, "scales alone")
    same(moe.swiglu(gu.to(DEV))[0], h, "h alone")


def test_swiglu_checkpoint_blocks():
    """Blocks over the whole range of fp32: zeros, -0, subnormal, tiny and huge maxima, ties."""
    rows, I = 64, 256
    gu = rnd(rows, 2 * I) * torch.logspace(-44, 37, rows)[:, None]
    gu[0] = 0
    gu[1] = -0.0
    gu[2, ::3] = 0
    gu[3] = torch.arange(2 * I).float() * 2.0 ** -140
    gu[4] = 448.0
    gu[4, ::2] = torch.arange(I).float() / 16  # quotients on and around the codes' midpoints
    gu[5] = (torch.arange(2 * I) % 128 - 64).float() * (448 / 64)
    gu[6, 1] = 3.4e38
    q, s = moe.swiglu(gu.to(DEV), checkpoint=True)[3:]
    cq, cs = oracle.quantize_fp8(gu, "f32")
    assert np.array_equal(s.cpu().numpy(), cs), "scales"
    assert np.array_equal(bits(q).numpy().reshape(cq.shape), cq), "codes"


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,I", [s for s in SWIGLU if s[1] % 128 == 0])
def test_swiglu_backward(rows, I, dt):
    gu, dh = outliers(rows, 2 * I, dt=dt), rnd(rows, I, seed=5, scale=1e-2, dt=dt)
    q, s = moe.quantize_fp8(gu.to(DEV))
    g = Guarded()
    d, h = moe.swiglu_backward(dh.to(DEV), q, s, want_h=True, out=(g((rows, 2 * I), dt), g((rows, I), dt)))
    g.check()
    kept = ref.values(q.cpu(), s.cpu())
    want, size = ref.swiglu_backward(dh, kept)
    rel = silu_rel(kept[:, :I]) + 8 * EPS32
    floor = 2.0 ** -125 * (1 + kept.abs().amax() ** 2)
    within(d, want, want.abs() * half_step(dt) + 1.01 * size * rel.repeat(1, 2) + floor, "d_gu")
    wh = ref.swiglu(kept)
    within(h, wh, wh.abs() * (half_step(dt) + 1.01 * rel) + floor, "h")
    a = dh.to(DEV).clone()
    d2, h2 = moe.swiglu_backward(a, q, s, want_h=True, out=(None, a))
    same(d, d2, "d_gu, h over dh")
    same(h, h2, "h over dh")
    same(moe.swiglu_backward(dh.to(DEV), q, s)[0], d, "d_gu alone")


def test_swiglu_backward_against_differences():
    rows, I = 4, 128
    q, s = moe.quantize_fp8(rnd(rows, 2 * I).to(DEV))
    kept, dh = ref.values(q.cpu(), s.cpu()), rnd(rows, I, seed=1)
    d = moe.swiglu_backward(dh.to(DEV), q, s)[0].cpu().to(F64)
    for seed in range(4):
        v = rnd(rows, 2 * I, seed=10 + seed).to(F64)
        a = ref.differences(lambda x: (ref.swiglu(x) * dh.to(F64)).sum(), kept, v, 1e-5)
        assert abs(float((d * v).sum()) - a) < 1e-3  # a thousand terms of order 1, 2^-20 each


def test_swiglu_saturated_gates():
    """Gates whose exponentials leave fp32's range give the limits, not NaN."""
    I = 128
    gate = torch.tensor([-3e38, -1e4, -200.0, -100.0, -88.0, 0.0, -0.0, 88.0, 100.0, 1e4, 1e18])
    gu = torch.zeros(len(gate), 2 * I)
    gu[:, :I] = gate[:, None]
    gu[:, I:] = 2.0
    for dt in TYPES:
        a = gu.to(dt)
        h = moe.swiglu(a.to(DEV))[0].cpu()
        want = ref.swiglu(a)
        within(h, want, want.abs() * (half_step(dt) + silu_rel(a[:, :I].to(F64).clamp(-100, 100))) + 2.0 ** -118, "h")
        q, s = moe.quantize_fp8(a.to(DEV))
        d = moe.swiglu_backward(torch.ones(len(gate), I, dtype=dt, device=DEV), q, s)[0].cpu()
        assert bool(d.isfinite().all())


# ------------------------------------------------------------------ alignment
def shifted(t):
    """The same values at an address that is one element past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    buf[1:] = t.reshape(-1).to(DEV)
    return buf[1:].view(t.shape)


def test_elements_alone_aligned():
    """Scales, ids, places and logits need only their element's alignment."""
    T, H, E, k, I = 37, 256, 16, 3, 128
    up = spread(T, E, k)
    x, w, l, sc = rnd(T, H).to(DEV), torch.ones(H, device=DEV), rnd(T, E), rnd(T, k, seed=1)
    ids = l.topk(k, 1).indices.int()
    ys = shifted(torch.zeros(T, H // 128))
    want = moe.rmsnorm(x, w, quantize=True)
    got = moe.rmsnorm(x, w, quantize=True, out=(None, None, None, ys))
    assert got[3].data_ptr() % 16 == 4
    same(got[3], want[3], "y_scale")
    rs = shifted(torch.zeros(T * k, H // 128))
    a, b = moe.dispatch(want[2], shifted(up), k, x_scale=shifted(want[3].cpu()), out=(None, rs)), \
        moe.dispatch(want[2], up.to(DEV), k, x_scale=want[3])
    same(a[0], b[0], "rows")
    same(a[1], b[1], "rows_scale")
    rows = moe.dispatch(x, up.to(DEV), k)
    same(moe.dispatch_backward(rows, shifted(up), k), moe.dispatch_backward(rows, up.to(DEV), k), "dx")
    a = moe.finalize_backward(x, rows, shifted(up), shifted(sc), out=(None, shifted(torch.zeros(T, k))))
    b = moe.finalize_backward(x, rows, up.to(DEV), sc.to(DEV))
    same(a[0], b[0], "d_fc2")
    same(a[1], b[1], "d_scales")
    for method in range(7):
        same(moe.route_backward(shifted(l), shifted(ids), shifted(sc), method),
             moe.route_backward(l.to(DEV), ids.to(DEV), sc.to(DEV), method), f"d_logits, method {method}")
    gu = rnd(T, 2 * I, seed=3).to(DEV)
    want = moe.swiglu(gu, quantize=True, checkpoint=True, want_h=True)
    got = moe.swiglu(gu, quantize=True, checkpoint=True, want_h=True,
                     out=(None, None, shifted(torch.zeros(T, 1)), None, shifted(torch.zeros(T, 2))))
    same(got[2], want[2], "h_scale")
    same(got[4], want[4], "gu_scale")
    same(moe.swiglu_backward(want[0], want[3], shifted(want[4].cpu()))[0],
         moe.swiglu_backward(want[0], want[3], want[4])[0], "d_gu")


# ------------------------------------------------------- empty calls, refusals
def test_no_rows():
    w = torch.ones(256, device=DEV)
    e, i = torch.empty(0, 256, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    s = torch.empty(0, 2, device=DEV)
    y, total, yq, ys = moe.rmsnorm(e, w, residual=e, quantize=True)
    assert y.shape == total.shape == yq.shape == (0, 256) and ys.shape == (0, 2)
    assert moe.dispatch(e, i, 2, 1).shape == (0, 256) and moe.dispatch_backward(e, i, 2, 1).shape == (0, 256)
    assert [t.shape for t in moe.finalize_backward(e, e, i, s, 1)] == [(0, 256), (0, 2)]
    assert moe.route_backward(e, i.view(0, 2), s, 1).shape == (0, 256)
    assert moe.swiglu(e, quantize=True, checkpoint=True)[1].shape == (0, 128)
    q = torch.empty(0, 512, dtype=F8, device=DEV)
    assert moe.swiglu_backward(e, q, torch.empty(0, 4, device=DEV))[0].shape == (0, 512)


def test_binding_refusals():
    x, w, i = torch.zeros(4, 256, device=DEV), torch.ones(256, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV)
    s = torch.zeros(4, 2, device=DEV)
    bad = [
        lambda: moe.rmsnorm(x, w.bfloat16()), lambda: moe.rmsnorm(x, w[:128]), lambda: moe.rmsnorm(x[0], w),
        lambda: moe.rmsnorm(x.t(), w), lambda: moe.rmsnorm(x.half(), w.half()),
        lambda: moe.rmsnorm(x, w, residual=x.bfloat16()), lambda: moe.rmsnorm(x, w, residual=x[:2]),
        lambda: moe.rmsnorm(x, w, out=(None, x, None, None)), lambda: moe.rmsnorm(x, w, out=(None, None, x, None)),
        lambda: moe.rmsnorm(x, w, residual=x.clone(), out=(x[:2], None, None, None)),
        lambda: moe.rmsnorm(x, w, quantize=True, want_y=False, out=(x, None, None, None)),
        lambda: moe.rmsnorm_backward(x[:2], x, w), lambda: moe.rmsnorm_backward(x.bfloat16(), x, w),
        lambda: moe.rmsnorm_backward(x, x, w, ws=w), lambda: moe.rmsnorm_backward(x, x, w, out=(None, w.bfloat16())),
        lambda: moe.dispatch(x, i, 3), lambda: moe.dispatch(x, i, 1), lambda: moe.dispatch(x, i.long(), 2),
        lambda: moe.dispatch(x, i, 2, x_scale=s), lambda: moe.dispatch(x.to(F8), i, 2),
        lambda: moe.dispatch(x, i, 0), lambda: moe.dispatch(x, i, 2, out=x),
        lambda: moe.dispatch_backward(x, i, 2, 1), lambda: moe.dispatch_backward(x, i, 3),
        lambda: moe.finalize_backward(x, x, i, s), lambda: moe.finalize_backward(x[:2], torch.zeros(8, 256, device=DEV), i, s),
        lambda: moe.route_backward(x, i, s, 0), lambda: moe.route_backward(x, i.view(4, 2), s[:, :1], 0),
        lambda: moe.route_backward(x.bfloat16(), i.view(4, 2), s, 0),
        lambda: moe.swiglu(torch.zeros(4, 255, device=DEV)), lambda: moe.swiglu(x, out=(None, x, None, None, None)),
        lambda: moe.swiglu_backward(x, x, s), lambda: moe.swiglu_backward(x, torch.zeros(4, 256, dtype=F8, device=DEV), s),
        lambda: moe.swiglu_backward(x, torch.zeros(4, 512, dtype=F8, device=DEV), s),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted:", n)
    big = torch.zeros(4 * 256 + 1, device=DEV)
    for call in (lambda: moe.rmsnorm(big[1:].view(4, 256), w), lambda: moe.rmsnorm(x, w, eps=0.0),
                 lambda: moe.rmsnorm(x[:, :100].contiguous(), w[:100]), lambda: moe.swiglu(x[:, :200].contiguous(), checkpoint=True),
                 lambda: moe.rmsnorm(x[:, :136].contiguous(), w[:136], quantize=True),
                 lambda: moe.rmsnorm_backward(x, x, w, ws=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(moe.MoeError):
            call()


# ------------------------------------------------------ together, as used
E_, K_, H_, I_, SH_ = 8, 3, 256, 128, 1


def experts(dt=FP):
    G = E_ + SH_
    return (rnd(G, 2 * I_, H_, seed=50, scale=H_ ** -0.5, dt=dt), rnd(G, H_, I_, seed=51, scale=I_ ** -0.5, dt=dt),
            rnd(E_, H_, seed=52, scale=H_ ** -0.5))


def products(rows, offsets, w, transpose):
    """Each expert's rows times its matrix (a caller's own product)."""
    out = torch.empty((rows.shape[0], w.shape[1 if transpose else 2]), dtype=rows.dtype, device=rows.device)
    for g in range(w.shape[0]):
        a, b = int(offsets[g]), int(offsets[g + 1])
        out[a:b] = rows[a:b] @ (w[g].t() if transpose else w[g])
    return out


def train_step(x, r, wn, w13, w2, wg, dy):
    """One training step of the layer from the library's operators and a caller's products."""
    y, total, _, _ = moe.rmsnorm(x, wn, 1e-5, residual=r)
    logits = y @ wg.t()
    ids, scales = moe.route(logits, K_, 2, 4, 2, None, 2.5)
    off, pair, up = moe.permute(ids, E_, SH_)
    rows = moe.dispatch(y, up, K_, SH_)
    offs = off.cpu()
    gu = products(rows, offs, w13, True)
    h, _, _, gq, gs = moe.swiglu(gu, checkpoint=True)
    fc2 = products(h, offs, w2, True)
    out = moe.finalize(fc2, up, scales, SH_)
    d_fc2, d_scales = moe.finalize_backward(dy, fc2, up, scales, SH_)
    dh = products(d_fc2, offs, w2, False)
    d_gu, h2 = moe.swiglu_backward(dh, gq, gs, want_h=True)
    d_rows = products(d_gu, offs, w13, False)
    d_logits = moe.route_backward(logits, ids, d_scales, 2, 2.5)
    d_y = moe.dispatch_backward(d_rows, up, K_, SH_) + d_logits @ wg
    dz, dwn = moe.rmsnorm_backward(d_y, total, wn, 1e-5, dsum=dy)
    G = E_ + SH_
    dw2 = torch.stack([d_fc2[int(offs[g]):int(offs[g + 1])].t() @ h2[int(offs[g]):int(offs[g + 1])] for g in range(G)])
    dw13 = torch.stack([d_gu[int(offs[g]):int(offs[g + 1])].t() @ rows[int(offs[g]):int(offs[g + 1])] for g in range(G)])
    return dict(out=out, dz=dz, dwn=dwn, dw2=dw2, dw13=dw13, dwg=d_logits.t() @ y), (ids, up, off, gq, gs)


def test_training_step():
    """norm, routing, rows to the experts, activation with its checkpoint, and all of it back, against
    the same step in 64 bits (with the step's own choice of experts and checkpoint)."""
    T = 75
    x, r, wn, dy = rnd(T, H_), rnd(T, H_, seed=1), 1 + 0.1 * rnd(H_, seed=2), rnd(T, H_, seed=3, scale=1e-2)
    w13, w2, wg = experts()
    dev = [t.to(DEV) for t in (x, r, wn, w13, w2, wg, dy)]
    got, (ids, up, off, gq, gs) = train_step(*dev)
    again, _ = train_step(*dev)
    for n in got:
        same(got[n], again[n], f"{n} again")
    # 64 bits
    e = float(np.float32(1e-5))
    z = (x + r).to(F64)
    y = ref.rmsnorm(z, wn, e)
    logits = y @ wg.to(F64).t()
    ids, up, offs = ids.cpu(), up.cpu(), off.cpu()
    scales = ref.route_scales(logits, ids, 2, 2.5, False)
    rows = ref.dispatch(y, up, K_, SH_)
    gu = products(rows, offs, w13.to(F64), True)
    fc2 = products(ref.swiglu(gu), offs, w2.to(F64), True)
    want = dict(out=ref.finalize(fc2, up, scales, SH_))
    d64 = dy.to(F64)
    d_fc2 = ref.dispatch(d64, up, K_, SH_)
    d_fc2[up.long()] *= scales.reshape(-1, 1)
    d_scales = (d64[:, None] * fc2[up.long()].view(T, K_, H_)).sum(2)
    kept = ref.values(gq.cpu(), gs.cpu())
    within(kept, gu, ref.code_tolerance(gu, gs.cpu()) * 1.01 + gu.abs() * 1e-3, "checkpoint")
    d_gu, _ = ref.swiglu_backward(products(d_fc2, offs, w2.to(F64), False), kept)
    d_logits, _ = ref.route_backward(logits, ids, d_scales, 2, 2.5, False)
    d_y = ref.dispatch_backward(products(d_gu, offs, w13.to(F64), False), up, K_, SH_)[0] + d_logits @ wg.to(F64)
    want["dz"], want["dwn"], _, _ = ref.rmsnorm_backward(d_y, z, wn, e, d64)
    h2 = ref.swiglu(kept)
    G = E_ + SH_
    want["dw2"] = torch.stack([d_fc2[int(offs[g]):int(offs[g + 1])].t() @ h2[int(offs[g]):int(offs[g + 1])] for g in range(G)])
    want["dw13"] = torch.stack([d_gu[int(offs[g]):int(offs[g + 1])].t() @ rows[int(offs[g]):int(offs[g + 1])] for g in range(G)])
    want["dwg"] = d_logits.t() @ y
    for n, v in want.items():
        off_by = float((got[n].cpu().to(F64) - v).norm() / v.norm())
        # a dozen fp32 steps in a row, the products' sums of 128 to 256 terms the longest of them
        assert off_by < 2e-5, (n, off_by)


@pytest.mark.parametrize("fused", [False, True])
def test_norm_feeds_the_fp8_layer(fused):
    """rmsnorm's codes and scales are the fp8 layer's input: no quantise step between them."""
    T, H, I, E, k = 70, 256, 128, 16, 4
    w8 = lambda t: t.to(F8)  # noqa: E731
    x, r, wn = rnd(T, H, dt=BF).to(DEV), rnd(T, H, seed=1, dt=BF).to(DEV), torch.ones(H, dtype=BF, device=DEV)
    w13, w2 = w8(rnd(E, 2 * I, H, seed=2)).to(DEV), w8(rnd(E, H, I, seed=3)).to(DEV)
    s13, s2 = torch.full((E, 2 * I // 128, H // 128), 0.06, device=DEV), torch.full((E, H // 128, I // 128), 0.09, device=DEV)
    y, total, yq, ys = moe.rmsnorm(x, wn, residual=r, quantize=True)
    logits = (y.float() @ rnd(E, H, seed=4).to(DEV).t()).contiguous()
    layer = moe.MoELayer(T, H, I, E, k, moe.ROUTE_RENORMALIZE, device=DEV, fp8_act=True, fused=fused)
    got = layer(y, logits, w13, w2, w13_scale=s13, w2_scale=s2, codes=(yq, ys)).clone()
    ids, sc = moe.route(logits, k, moe.ROUTE_RENORMALIZE)
    off, pair, up = moe.permute(ids, E)
    want = moe.finalize(moe.expert_ffn_fp8(yq, ys, off, pair, w13, w2, s13, s2, k, E), up, sc)
    same(got, want, "layer from the norm's codes")
    with pytest.raises(ValueError, match="fp8"):
        moe.MoELayer(T, H, I, E, k, moe.ROUTE_RENORMALIZE, device=DEV)(y, logits, w13, w2, codes=(yq, ys))


def test_side_stream_and_graph():
    """The operators on a stream of their own, then captured in two graphs that share a workspace and
    replayed in turn between eager calls: every replay equals the eager result."""
    T, H, E, k, I = 130, 512, 16, 4, 256
    up = spread(T, E, k).to(DEV)
    sets = []
    for seed in (0, 100):
        sets.append(dict(x=rnd(T, H, seed=seed, dt=BF).to(DEV), r=rnd(T, H, seed=seed + 1, dt=BF).to(DEV),
                         w=rnd(H, seed=seed + 2, dt=BF).to(DEV), l=rnd(T, E, seed=seed + 3).to(DEV),
                         s=rnd(T, k, seed=seed + 4).to(DEV), gu=rnd(T * k, 2 * I, seed=seed + 5, dt=BF).to(DEV),
                         rows=rnd(T * k, H, seed=seed + 6, dt=BF).to(DEV)))
        sets[-1]["ids"] = sets[-1]["l"].topk(k, 1).indices.int()
    ws = moe.rmsnorm_backward_workspace(T, H)

    def all_of(c):
        out = [*moe.rmsnorm(c["x"], c["w"], residual=c["r"], quantize=True)]
        out += moe.rmsnorm_backward(c["r"], c["x"], c["w"], dsum=c["r"], ws=ws)
        out += [moe.dispatch(c["x"], up, k), moe.dispatch_backward(c["rows"], up, k)]
        out += moe.finalize_backward(c["x"], c["rows"], up, c["s"])
        out += [moe.route_backward(c["l"], c["ids"], c["s"], 0), moe.route_backward(c["l"], c["ids"], c["s"], 2)]
        h, hq, hs, q, qs = moe.swiglu(c["gu"], quantize=True, checkpoint=True, want_h=True)
        out += [h, hq, hs, q, qs, *moe.swiglu_backward(h, q, qs, want_h=True)]
        return out

    eager = [[t.clone() for t in all_of(c)] for c in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_of(sets[0])
    side.synchronize()
    for n, (a, b) in enumerate(zip(got, eager[0])):
        same(a, b, f"output {n} on a side stream")
    graphs = []
    for c in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, all_of(c)))
    for turn in range(4):
        for i, (g, out) in enumerate(graphs):
            for t in out:
                t.view(torch.uint8).fill_(0x5A)
            g.replay()
            torch.cuda.synchronize()
            for n, (a, b) in enumerate(zip(out, eager[i])):
                same(a, b, f"graph {i}, replay {turn}, output {n}")
            all_of(sets[1 - i])


def test_timing_names_every_kernel():
    T, H, k = 8, 256, 2
    up = spread(T, 4, k).to(DEV)
    x, w, s = rnd(T, H).to(DEV), torch.ones(H, device=DEV), rnd(T, k).to(DEV)
    binding.timing_enable(True)
    try:
        binding.kernel_times(reset=True)
        moe.rmsnorm(x, w)
        moe.rmsnorm_backward(x, x, w)  # few rows: one kernel
        big = x.repeat(32, 1)
        moe.rmsnorm_backward(big, big, w)
        rows = moe.dispatch(x, up, k)
        moe.dispatch_backward(rows, up, k)
        moe.finalize_backward(x, rows, up, s)
        moe.route_backward(x, up.view(T, k), s, 1)
        q = moe.swiglu(x, checkpoint=True)
        moe.swiglu_backward(q[0], q[3], q[4])
        t = binding.kernel_times(reset=True)
    finally:
        binding.timing_enable(False)
    for name, n in (("rmsnorm", 1), ("rmsnorm_backward", 2), ("rmsnorm_dweight", 1), ("dispatch", 1),
                    ("dispatch_backward", 1), ("finalize_backward", 1), ("route_backward", 1), ("swiglu", 1),
                    ("swiglu_backward", 1)):
        assert t[name][1] == n and t[name][0] > 0, name
