"""The layer for few tokens on the GPU.

The routing is compared bit for bit with moe_route.  The rest is held to 64 bits in two parts: the h
that the call leaves in its workspace against h of the exact inputs (the fp32 work and one rounding),
and y against the weighted sum of FC2 rows of that h (the fp32 work and one rounding)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_07_amd as moe
import mxfp4_ref
import oracle
from mixture_experts_layer_07_amd import binding
from rowops_ref import EPS32, F64, half_step
from test_gpu_rowops import BF, DEV, F8, FP, Guarded, bits, rnd, same, within

pytestmark = pytest.mark.gpu

Q4, S8, U8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu, torch.uint8
WDT = ["f32", "bf16", "fp8", "mxfp4"]
DEFAULT, RENORM, DSV3, LLAMA4, NAIVE, MINIMAX2, SIGMOID = range(7)
# K values that one matrix instruction adds
STEP = dict(f32=4, bf16=32, fp8=32, mxfp4=32)


def matrices(G, N, K, wdt, seed):
    """(weights, scales or None, their values in 64 bits)"""
    v = rnd(G * N, K, seed=seed, scale=K ** -0.5)
    if wdt == "f32":
        return v.view(G, N, K), None, v.to(F64).view(G, N, K)
    if wdt == "bf16":
        return v.to(BF).view(G, N, K), None, v.to(BF).to(F64).view(G, N, K)
    if wdt == "fp8":
        b = v.view(G, N // 128, 128, K // 128, 128)
        s = b.abs().amax((2, 4)) / 448 * torch.from_numpy(np.random.default_rng(seed).uniform(0.8, 1.2, (G, N // 128, K // 128))).float()
        q = (b / s[:, :, None, :, None]).clamp(-448, 448).to(F8)
        return q.view(G, N, K), s, (q.float().to(F64) * s.to(F64)[:, :, None, :, None]).view(G, N, K)
    c, s = mxfp4_ref.encode(v)
    p = mxfp4_ref.pack(c)
    return p.view(Q4).view(G, N, K // 2), s.view(S8).view(G, N, K // 32), mxfp4_ref.decode(p, s).view(G, N, K)


class Layer:
    def __init__(self, T, H, I, E, k, wdt, n_shared=0, method=RENORM, seed=0, logits=None, **routing):
        self.T, self.H, self.I, self.E, self.k, self.wdt, self.sh = T, H, I, E, k, wdt, n_shared
        self.dt = FP if wdt == "f32" else BF
        self.x = rnd(T, H, seed=seed)
        self.x[:, ::61] *= 9
        self.x = self.x.to(self.dt)
        self.logits = rnd(T, E, seed=seed + 1) if logits is None else logits
        self.method, self.routing = method, routing
        G = E + n_shared
        self.w13, self.s13, self.d13 = matrices(G, 2 * I, H, wdt, seed + 2)
        self.w2, self.s2, self.d2 = matrices(G, H, I, wdt, seed + 3)

    def gpu(self):
        d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        r = {n: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for n, v in self.routing.items()}
        return dict(x=d(self.x), logits=d(self.logits), w13=d(self.w13), w2=d(self.w2), k=self.k, method=self.method,
                    w13_scale=d(self.s13), w2_scale=d(self.s2), n_shared=self.sh, **r)

    def run(self, **change):
        out = Guarded()
        a = dict(self.gpu(), **change)
        T = a["x"].shape[0]
        bufs = out((T, self.H), self.dt), out((T, self.k), torch.int32), out((T, self.k), FP)
        n = moe.layer_few_workspace(T, self.H, self.I, self.E, self.k, self.sh, self.dt).numel()
        ws = out((n,), U8)
        got = moe.layer_few(**a, ws=ws, out=bufs)
        assert all(p is q for p, q in zip(got, bufs))
        out.check()
        h = ws[:T * (self.k + self.sh) * self.I * bufs[0].element_size()]
        return got, h.view(self.dt).view(-1, self.I)

    def check(self):
        (y, ids, scales), h = self.run()
        g = self.gpu()
        want = moe.route(g["logits"], self.k, self.method, **{n: v for n, v in self.routing_gpu(g).items()})
        same(ids, want[0], "ids")
        same(scales, want[1], "scales")
        ids, scales, h, y = ids.cpu(), scales.cpu().to(F64), h.cpu().to(F64), y.cpu()
        T, k, I = self.T, self.k, self.I
        _, pair, up = oracle.permute(ids.numpy(), self.E, self.sh)
        x = self.x.to(F64)
        total, size = torch.zeros(T, self.H, dtype=F64), torch.zeros(T, self.H, dtype=F64)

        def rows(e, tok, at, weight):
            w13, w2 = self.d13[e], self.d2[e]
            gu, s = x[tok] @ w13.t(), x[tok].abs() @ w13.abs().t()
            # each instruction's sums are good to two half-steps of what has been added, then the waves' sums
            err = (2 * self.H / STEP[self.wdt] + 16) * EPS32 * s
            gt, u = gu[:, :I], gu[:, I:]
            sig = torch.sigmoid(gt)
            hv = gt * sig * u
            slope = (sig * (1 + gt * (1 - sig))).abs()
            off = (u.abs() + err[:, I:]) * (slope + 0.5 * err[:, :I]) * err[:, :I] + (gt * sig).abs() * err[:, I:]
            within(h[at], hv, (hv.abs() + off) * half_step(self.dt) + off + 16 * EPS32 * hv.abs() + 1e-37, f"h of expert {e}")
            total[tok] += weight[:, None] * (h[at] @ w2.t())
            size[tok] += weight.abs()[:, None] * (h[at].abs() @ w2.abs().t())

        up = torch.from_numpy(np.asarray(up)).long().view(T, k)
        for e in sorted(set(ids.flatten().tolist())):
            tok, j = (ids == e).nonzero(as_tuple=True)
            rows(e, tok, up[tok, j], scales[tok, j])
        for i in range(self.sh):
            tok = torch.arange(T)
            rows(self.E + i, tok, T * k + i * T + tok, torch.ones(T, dtype=F64))
        chain = 2 * self.I / STEP[self.wdt] + k + self.sh + 16
        within(y, total, total.abs() * half_step(self.dt) + chain * EPS32 * size + 1e-37, "y")

    def routing_gpu(self, g):
        return {n: g[n] for n in self.routing}


@pytest.mark.parametrize("wdt", WDT)
@pytest.mark.parametrize("T,H,I,E,k,sh", [(1, 128, 128, 8, 2, 0), (1, 1024, 256, 64, 8, 1), (13, 256, 512, 8, 2, 0),
                                          (2, 384, 640, 12, 3, 2), (7, 512, 1024, 100, 8, 0), (16, 640, 384, 33, 5, 1),
                                          (17, 256, 128, 256, 6, 1), (32, 128, 256, 256, 8, 2), (32, 256, 128, 2, 2, 1),
                                          (31, 128, 384, 1, 1, 0), (5, 2048, 128, 16, 1, 0)])
def test_layer(T, H, I, E, k, sh, wdt):
    Layer(T, H, I, E, k, wdt, sh, seed=T).check()


@pytest.mark.parametrize("wdt", WDT)
def test_long_rows(wdt):
    """Several pieces a wave and an odd number of them, in both products."""
    Layer(3, 7168, 256, 8, 2, wdt, 1).check()
    Layer(3, 256, 4224, 4, 2, wdt, 0).check()


@pytest.mark.parametrize("T", range(1, 33))
def test_every_token_count(T):
    Layer(T, 128, 128, 16, 3, "bf16", 1, seed=T).check()


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("method", range(7))
def test_methods(method, renormalize):
    E, T = 64, 6
    how = dict(scaling=2.5, renormalize=renormalize)
    if method in (DSV3, MINIMAX2):
        how["bias"] = rnd(E, seed=9, scale=0.1)
    if method == DSV3:
        how.update(n_group=8, topk_group=4)
    Layer(T, 256, 128, E, 8, "bf16", 1, method=method, **how).check()


def test_groups_that_are_no_power_of_two():
    Layer(9, 128, 128, 60, 4, "fp8", 0, method=DSV3, n_group=5, topk_group=2, scaling=2.5).check()


def test_equal_logits_and_infinities():
    """Ties go to the lowest experts, so every token shares them; masked experts are never chosen."""
    Layer(20, 128, 128, 40, 4, "bf16", logits=torch.zeros(20, 40)).check()
    l = rnd(20, 40, seed=1)
    l[:, ::2] = float("-inf")
    l[3, 1::2] = torch.finfo(FP).min
    Layer(20, 128, 128, 40, 4, "bf16", logits=l).check()


# the I whose rows give every wave as many pieces, where one workgroup has a column of y alone (H
# past 2048): y's order of summation is the token's own
EVEN_I = [("f32", 512), ("bf16", 1024), ("fp8", 1024), ("mxfp4", 2048)]


@pytest.mark.parametrize("wdt,I", EVEN_I)
def test_a_token_alone(wdt, I):
    """ids, weights and h of a token are the same alone and among others, and so is y at these I."""
    a = Layer(19, 2176, I, 5, 2, wdt, 1)
    (y, ids, scales), h = a.run()
    g = a.gpu()
    _, _, up = oracle.permute(ids.cpu().numpy(), a.E, 1)
    up = torch.from_numpy(np.asarray(up)).view(19, 2)
    for t in (0, 7, 18):
        (y1, i1, s1), h1 = a.run(x=g["x"][t:t + 1].clone(), logits=g["logits"][t:t + 1].clone())
        same(i1[0], ids[t], "ids")
        same(s1[0], scales[t], "scales")
        own = ids[t].cpu().argsort()
        same(h1[:2], h[up[t][own].long().to(DEV)], "h")
        same(h1[2], h[19 * 2 + t], "shared h")
        same(y1[0], y[t], "y")


@pytest.mark.parametrize("wdt,I", EVEN_I)
def test_nan_stays_with_its_token(wdt, I):
    a = Layer(12, 2176, I, 4, 2, wdt, 1)
    (clean, ids, _), _ = a.run()
    bad = a.x.clone()
    bad[5, 17] = float("nan")
    bad[6, 3] = float("inf")
    (y, i2, _), _ = a.run(x=bad.to(DEV))
    same(i2, ids, "ids")
    rest = [t for t in range(12) if t not in (5, 6)]
    same(y[rest], clean[rest], "other tokens")
    assert bool(y[5].isnan().all()) and not bool(y[6].isfinite().all())
    l = a.logits.clone()
    l[2] = float("nan")  # any experts, no other token's result
    (y, i3, _), _ = a.run(logits=l.to(DEV))
    rest = [t for t in range(12) if t != 2]
    same(y[rest], clean[rest], "other tokens")
    assert bool(((i3 >= 0) & (i3 < 4)).all())


def test_a_token_with_every_expert_masked():
    """moe_route's ids and weights for it, and the other tokens' results as they were."""
    a = Layer(9, 2176, 1024, 8, 4, "bf16")
    l = a.logits.clone()
    l[4] = float("-inf")
    for a.method in range(7):
        (clean, _, _), _ = a.run()
        g = dict(a.gpu(), logits=l.to(DEV))
        (y, ids, scales), _ = a.run(logits=g["logits"])
        want = moe.route(g["logits"], 4, a.method)
        same(ids, want[0], "ids")
        same(scales, want[1], "scales")
        rest = [t for t in range(9) if t != 4]
        same(y[rest], clean[rest], "other tokens")


def test_weights_that_no_token_chooses_are_not_read():
    """NaN in every other expert changes nothing."""
    a = Layer(2, 128, 128, 16, 2, "bf16")
    (clean, ids, _), _ = a.run()
    chosen = set(ids.flatten().tolist())
    w13, w2 = a.w13.clone(), a.w2.clone()
    for e in set(range(16)) - chosen:
        w13[e] = w2[e] = float("nan")
    (y, _, _), _ = a.run(w13=w13.to(DEV), w2=w2.to(DEV))
    same(y, clean, "y")


@pytest.mark.parametrize("wdt", WDT)
def test_against_the_separate_calls(wdt):
    """The same layer through route, permute, FFN and finalize (MXFP4 weights: their bf16 values)."""
    a = Layer(11, 512, 256, 16, 4, wdt, 1)
    g = a.gpu()
    (y, _, _), _ = a.run()
    ids, scales = moe.route(g["logits"], 4, RENORM)
    off, pair, up = moe.permute(ids, 16, 1)
    w = (g["w13"], g["w2"])
    s = (g["w13_scale"], g["w2_scale"])
    if wdt == "mxfp4":
        w = [moe.dequantize_mxfp4(q.view(-1, q.shape[2]), t.view(-1, t.shape[2])).view(q.shape[0], q.shape[1], -1)
             for q, t in zip(w, s)]
        s = (None, None)
    rows = moe.expert_ffn(g["x"], off, pair, w[0], w[1], 4, 16, 1, *s)
    want = moe.finalize(rows, up, scales, 1)
    far = float((y.double() - want.double()).norm() / want.double().norm())
    # FC2's rows are rounded there and not here, y and h in both
    assert far < (3 * half_step(BF) if a.dt == BF else 1e-6), far


def test_layer_object():
    for wdt in WDT:
        a = Layer(6, 256, 128, 8, 2, wdt, 1, method=DEFAULT, renormalize=True)
        g = a.gpu()
        layer = moe.MoELayer(6, 256, 128, 8, 2, DEFAULT, a.dt, renormalize=True, n_shared=1, few=True)
        y = layer(g["x"], g["logits"], g["w13"], g["w2"], None, g["w13_scale"], g["w2_scale"])
        (want, ids, scales), _ = a.run()
        same(y, want, "y")
        same(layer.ids, ids, "ids")
        same(layer.scales, scales, "scales")
        with pytest.raises(ValueError, match="codes"):
            layer(g["x"], g["logits"], g["w13"], g["w2"], codes=(y, y))
    for bad in (dict(T=33, few=True), dict(few=True, mxfp4=True), dict(few=True, fp8_act=True), dict(few=True, fused=True),
                dict(mxfp4=True, fp8_act=True), dict(mxfp4=True, fused=True), dict(mxfp4=True, act_dtype=FP)):
        with pytest.raises(ValueError):
            moe.MoELayer(**{**dict(T=6, H=256, I=128, E=8, k=2, method=0), **bad})


@pytest.mark.parametrize("codes", [False, True])
def test_layer_object_mxfp4(codes):
    """The 4-bit layer: prefill rows through expert_ffn_mxfp4, a few of the tokens through layer_few."""
    a = Layer(40, 256, 256, 8, 2, "mxfp4", 1)
    g = a.gpu()
    layer = moe.MoELayer(40, 256, 256, 8, 2, RENORM, n_shared=1, mxfp4=True)
    given = moe.quantize_mxfp4(g["x"]) if codes else None
    y = layer(None if codes else g["x"], g["logits"], g["w13"], g["w2"], None, g["w13_scale"], g["w2_scale"], codes=given)
    xq, xs = moe.quantize_mxfp4(g["x"])
    ids, scales = moe.route(g["logits"], 2, RENORM)
    off, pair, up = moe.permute(ids, 8, 1)
    rows = moe.expert_ffn_mxfp4(xq, xs, off, pair, g["w13"], g["w2"], g["w13_scale"], g["w2_scale"], 2, 8, 1)
    same(y, moe.finalize(rows, up, scales, 1), "the separate calls")
    few = moe.MoELayer(3, 256, 256, 8, 2, RENORM, n_shared=1, few=True)
    z = few(g["x"][:3].contiguous(), g["logits"][:3].contiguous(), g["w13"], g["w2"], None, g["w13_scale"], g["w2_scale"])
    same(few.ids, layer.ids[:3], "ids")
    want, _, _ = moe.layer_few(g["x"][:3].contiguous(), g["logits"][:3].contiguous(), g["w13"], g["w2"], 2, RENORM,
                               g["w13_scale"], g["w2_scale"], n_shared=1)
    same(z, want, "y")


def test_repeats_side_stream_and_graphs():
    layers = [Layer(t, 512, 256, 32, 4, w, 1, method=DSV3, n_group=4, topk_group=2, seed=t)
              for t, w in ((1, "bf16"), (9, "fp8"), (20, "mxfp4"), (5, "f32"))]
    eager = [[t.clone() for t in a.run()[0]] for a in layers]
    for a, e in zip(layers, eager):
        for p, q in zip(a.run()[0], e):
            same(p, q, "again")
    ins = [a.gpu() for a in layers]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [moe.layer_few(**i) for i in ins]
    side.synchronize()
    for p, q in zip(got, eager):
        for m, n in zip(p, q):
            same(m, n, "side stream")
    ws = torch.empty(1 << 20, dtype=U8, device=DEV)
    graphs = []
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, moe.layer_few(**i, ws=ws)))
    for turn in range(4):
        for (g, out), want, other in zip(graphs, eager, ins[::-1]):
            for t in out:
                t.view(U8).fill_(0x5A)
            ws.fill_(0x5A)
            g.replay()
            torch.cuda.synchronize()
            for p, q in zip(out, want):
                same(p, q, f"replay {turn}")
            moe.layer_few(**other, ws=ws)


@pytest.mark.parametrize("H", [128, 512, 1024, 2048])
def test_workgroups_that_share_columns(H):
    """However they finish, they give the same bits; also with the workspace as another call left it."""
    a = Layer(32, H, 384, 24, 4, "bf16", 1)
    g = a.gpu()
    ws = moe.layer_few_workspace(32, H, 384, 24, 4, 1, BF)
    (want, _, _), _ = a.run()
    for i in range(100):
        if i % 10 == 0:
            ws.fill_(i)
        same(moe.layer_few(**g, ws=ws)[0], want, f"run {i}")


def test_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    layers = [Layer(20, 512, 384, 24, 4, "bf16", 1, seed=1), Layer(3, 256, 512, 16, 2, "mxfp4", 0, seed=2)]
    ins = [a.gpu() for a in layers]
    want = [moe.layer_few(**i) for i in ins]
    ws = [moe.layer_few_workspace(a.T, a.H, a.I, a.E, a.k, a.sh, a.dt) for a in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.layer_few(**ins[i], ws=ws[i]))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for out in g:
            for p, q in zip(out, w):
                same(p, q, "the streams")


def test_large_weights():
    """Experts past 2^32 bytes into the weights."""
    g = torch.Generator(device=DEV).manual_seed(0)
    E, H, I = 20, 8192, 14336
    w13 = torch.empty((E, 2 * I, H), dtype=BF, device=DEV)
    w2 = torch.empty((E, H, I), dtype=BF, device=DEV)
    for e in range(E):
        w13[e] = torch.randn((2 * I, H), generator=g, device=DEV) * H ** -0.5
        w2[e] = torch.randn((H, I), generator=g, device=DEV) * I ** -0.5
    x = torch.randn((3, H), generator=g, device=DEV).to(BF)
    logits = torch.full((3, E), -9.0, device=DEV)
    logits[:, E - 1], logits[0, 0], logits[1, 9], logits[2, E - 2] = 1.0, 0.5, 0.5, 0.5
    y, ids, sc = moe.layer_few(x, logits, w13, w2, 2, RENORM)
    assert ids.tolist() == [[E - 1, 0], [E - 1, 9], [E - 1, E - 2]]
    want = torch.zeros(3, H, dtype=F64, device=DEV)
    for t in range(3):
        for j in range(2):
            e = int(ids[t, j])
            gu = w13[e].double() @ x[t].double()
            h = torch.nn.functional.silu(gu[:I]) * gu[I:]
            want[t] += float(sc[t, j]) * (w2[e].double() @ h)
    far = float((y.double() - want).norm() / want.norm())
    assert far < 2 * half_step(BF), far  # h and y rounded


def test_offsets_past_2_31_in_one_expert():
    """w13 just under 4 GiB, the largest that is taken."""
    g = torch.Generator(device=DEV).manual_seed(0)
    H, I = 1024, (1 << 20) - 128
    w13 = torch.empty((1, 2 * I, H), dtype=BF, device=DEV).normal_(0, H ** -0.5, generator=g)
    w2 = torch.empty((1, H, I), dtype=BF, device=DEV).normal_(0, I ** -0.5, generator=g)
    x = torch.randn((2, H), generator=g, device=DEV).to(BF)
    y, _, sc = moe.layer_few(x, torch.zeros((2, 1), device=DEV), w13, w2, 1, RENORM)
    want = torch.zeros(2, H, dtype=F64, device=DEV)
    for at in range(0, I, 1 << 17):
        part = slice(at, min(at + (1 << 17), I))
        h = torch.nn.functional.silu(x.double() @ w13[0, :I][part].double().t()) * (x.double() @ w13[0, I:][part].double().t())
        want += h @ w2[0, :, part].double().t()
    far = float((y.double() - want).norm() / want.norm())
    assert far < 2 * half_step(BF), far  # h and y rounded


def test_empty_and_refusals():
    a = Layer(4, 256, 128, 8, 2, "bf16")
    g = a.gpu()
    y, ids, sc = moe.layer_few(**{**g, "x": g["x"][:0], "logits": g["logits"][:0]})
    assert y.shape == (0, 256) and ids.shape == (0, 2)
    many = dict(g, x=g["x"].repeat(9, 1)[:33].contiguous(), logits=g["logits"].repeat(9, 1)[:33].contiguous())
    with pytest.raises(moe.MoeError, match="32 tokens"):
        moe.layer_few(**many)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.layer_few(**g, ws=torch.empty(16, dtype=U8, device=DEV))
    with pytest.raises(moe.MoeError, match="fp32"):
        moe.layer_few(**dict(g, x=g["x"].float()))
    for name, bad in (("logits", g["logits"][:3]), ("logits", g["logits"].double()), ("x", g["x"].half()),
                      ("w13", g["w13"][0]), ("w13", g["w13"][:3]), ("w2", g["w2"][:, :128]), ("w2", g["w2"].float()),
                      ("bias", torch.zeros(3, device=DEV)), ("x", g["x"].t())):
        with pytest.raises(ValueError):
            moe.layer_few(**dict(g, **{name: bad}))
    q = Layer(4, 256, 128, 8, 2, "mxfp4").gpu()
    for name, bad in (("w13_scale", q["w13_scale"][:2]), ("w2_scale", q["w2_scale"].view(U8)), ("w13", q["w13"].view(U8))):
        with pytest.raises(ValueError):
            moe.layer_few(**dict(q, **{name: bad}))


def test_timing_names():
    a = Layer(4, 256, 128, 8, 2, "bf16").gpu()
    binding.timing_enable(True)
    try:
        binding.kernel_times(reset=True)
        moe.layer_few(**a)
        t = binding.kernel_times(reset=True)
    finally:
        binding.timing_enable(False)
    for n in ("few_fc1", "few_fc2"):
        assert t[n][1] == 1 and t[n][0] > 0
    assert t["route"][1] == 0
