"""The 4-bit microscaled format and the experts' FFN on it, on the GPU.

Codes, scales and their values are compared bit for bit with the 64-bit forms.  The FFN is held to
them in two parts, which needs no allowance for a code that falls on the other side of a border:
the codes of h that it leaves in its workspace have to come from values that the fp32 work may have
made of the true h, and the output has to be the product of those codes, up to the fp32 work and
half a step of bf16 for its one rounding."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_07_amd as moe
import mxfp4_ref as ref
import oracle
from mixture_experts_layer_07_amd import binding
from mxfp4_ref import F64
from rowops_ref import half_step
from test_gpu_rowops import BF, DEV, FP, Guarded, bits, rnd, same, within

pytestmark = pytest.mark.gpu

Q4, S8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
U8 = torch.uint8


def to_bytes(t):
    return t.view(U8).cpu()


# ------------------------------------------------------------------- codes
def hard(rows, cols, dt, seed=0):
    """Blocks of every size that the type has, values on and next to the borders, zeros."""
    rng = np.random.default_rng([seed, rows, cols])
    v = rng.standard_normal((rows, cols // 32, 32))
    grid = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9])
    on = rng.random(v.shape) < 0.3
    v = np.where(on, rng.choice(grid, v.shape) * rng.choice([-1, 1], v.shape), v)
    v *= np.exp2(rng.integers(-149, 124, v.shape[:2]))[:, :, None]
    v[rng.random(v.shape[:2]) < 0.1] = 0.0
    v[rng.random(v.shape) < 0.02] = -0.0
    t = torch.from_numpy(v.reshape(rows, cols)).float()
    near_ = torch.from_numpy(rng.integers(-1, 2, (rows, cols)).astype(np.int32))  # a neighbour in fp32
    t = torch.where(torch.from_numpy(rng.random((rows, cols)) < 0.1) & (t != 0),
                    (t.view(torch.int32) + near_).view(FP), t)
    return t.to(dt)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (7, 7168), (333, 1120), (64, 4096), (4099, 32), (2, 16416)])
def test_codes(rows, cols, dt):
    x = hard(rows, cols, dt)
    out = Guarded()
    q, s = out((rows, cols // 2), Q4), out((rows, cols // 32), S8)
    got = moe.quantize_mxfp4(x.to(DEV), out=(q, s))
    assert got[0] is q and got[1] is s
    out.check()
    c, want = ref.encode(x)
    assert torch.equal(to_bytes(s), want), "scales"
    assert torch.equal(to_bytes(q), ref.pack(c)), "codes"
    for vt in (BF, FP):
        v = out((rows, cols), vt)
        moe.dequantize_mxfp4(q, s, vt, out=v)
        out.check()
        same(v, ref.decode(ref.pack(c), want).to(vt), f"values in {vt}")  # every one a value of the type
    same(moe.dequantize_mxfp4(q, s), ref.decode(ref.pack(c), want).to(BF), "new buffers")


@pytest.mark.parametrize("dt", [BF, FP])
def test_every_code_and_scale(dt):
    """256 bytes of codes under each of the 256 scales."""
    codes = torch.arange(256, dtype=torch.int32).to(U8).repeat(256, 1)            # [256 scales, 512 values]
    scale = torch.arange(256, dtype=torch.int32).to(U8)[:, None].repeat(1, 16).contiguous()
    got = moe.dequantize_mxfp4(codes.to(DEV).view(Q4), scale.to(DEV).view(S8), dt).cpu()
    want = ref.decode(codes, scale).to(dt)  # past the range: infinity
    assert torch.equal(got.isnan(), want.isnan()) and bool(want[255].isnan().all())
    same(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0), "values")


@pytest.mark.parametrize("dt", [BF, FP])
def test_codes_of_blocks_that_are_not_finite(dt):
    x = rnd(6, 256, dt=dt)
    clean = moe.quantize_mxfp4(x.to(DEV))
    bad = x.clone()
    bad[1, 40] = float("nan")
    bad[2, 95], bad[2, 96] = float("inf"), float("-inf")
    bad[4, 0:32] = float("nan")
    q, s = moe.quantize_mxfp4(bad.to(DEV))
    hit = torch.zeros(6, 8, dtype=torch.bool)
    hit[1, 1] = hit[2, 2] = hit[2, 3] = hit[4, 0] = True
    assert bool((to_bytes(s)[hit] == 255).all())
    assert torch.equal(to_bytes(s)[~hit], to_bytes(clean[1])[~hit])
    keep = (~hit).repeat_interleave(16, 1)
    assert torch.equal(to_bytes(q)[keep], to_bytes(clean[0])[keep])
    for vt in (BF, FP):
        v = moe.dequantize_mxfp4(q, s, vt).cpu()
        assert torch.equal(v.isnan(), hit.repeat_interleave(32, 1))


def test_codes_past_the_largest_grid():
    """More values than a launch has threads for, and arrays past 2^32 bytes: the parts of a large
    call are those parts' own calls."""
    cols = 8192
    rows = (1 << 33) // cols + 5
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((rows, cols), device=DEV)
    for a in range(0, rows, 1 << 16):
        x[a:a + (1 << 16)] = torch.randn((min(1 << 16, rows - a), cols), generator=g, device=DEV)
    q, s = moe.quantize_mxfp4(x)
    v = moe.dequantize_mxfp4(q, s, FP)
    for a, b in ((0, 3), ((1 << 32) // cols - 2, (1 << 32) // cols + 2), ((1 << 33) // cols - 2, rows)):
        pq, ps = moe.quantize_mxfp4(x[a:b].clone())
        same(q.view(U8)[a:b], pq.view(U8), "codes")
        same(s.view(U8)[a:b], ps.view(U8), "scales")
        same(v[a:b], moe.dequantize_mxfp4(pq, ps, FP), "values")


def test_empty_and_refusals():
    q, s = moe.quantize_mxfp4(torch.empty((0, 64), device=DEV))
    assert q.shape == (0, 32) and s.shape == (0, 2) and moe.dequantize_mxfp4(q, s).shape == (0, 64)
    x = torch.zeros((4, 64), device=DEV, dtype=BF)
    q, s = moe.quantize_mxfp4(x)
    with pytest.raises(moe.MoeError, match="multiple of 32"):
        moe.quantize_mxfp4(torch.zeros((4, 48), device=DEV))
    with pytest.raises(ValueError, match="multiple of 32"):
        moe.dequantize_mxfp4(q[:, :24].contiguous(), s)
    with pytest.raises(ValueError, match="contiguous"):
        moe.quantize_mxfp4(x.t())
    with pytest.raises(ValueError, match="dtype"):
        moe.quantize_mxfp4(x.half())
    with pytest.raises(ValueError, match="dtype"):
        moe.dequantize_mxfp4(q, s, torch.float16)
    with pytest.raises(ValueError, match="shape"):
        moe.dequantize_mxfp4(q, s[:2])
    with pytest.raises(ValueError, match="dtype"):
        moe.dequantize_mxfp4(q.view(U8), s)
    with pytest.raises(ValueError, match="rows, columns"):
        moe.quantize_mxfp4(x.view(2, 2, 64))
    with pytest.raises(moe.MoeError, match="aligned"):
        moe.quantize_mxfp4(torch.zeros(33 * 4, device=DEV)[1:129].view(4, 32))


# -------------------------------------------------------------------- FFN
class Case:
    """Inputs of one call, on the host in 64 bits and on the GPU."""

    def __init__(self, counts, H, I, n_shared=0, T=None, seed=0, k=None, alike=False):
        E = len(counts)
        P = sum(counts)
        rng = np.random.default_rng([seed, H, I, E, P])
        if k is None:
            k = 1
        T = P // k if T is None else T
        assert T * k == P
        self.T, self.H, self.I, self.E, self.k, self.sh = T, H, I, E, k, n_shared
        self.x = rnd(T, H, seed=seed)
        self.x[:, ::61] *= 9
        self.x *= torch.from_numpy(np.exp2(rng.integers(-3, 4, (T, 1)))).float()
        pair = rng.permutation(P).astype(np.int32)
        self.pair = torch.from_numpy(pair)
        self.offsets = torch.from_numpy(np.concatenate(
            [[0], np.cumsum(counts), P + T * np.arange(1, n_shared + 1)]).astype(np.int32))
        G = E + n_shared
        n = 1 if alike else G  # alike: every expert has the same weights
        q = lambda rows, cols, sd: [t.reshape(n, rows, -1).expand(G, -1, -1).contiguous()  # noqa: E731
                                    for t in self._weights(n * rows, cols, sd)]
        (self.w13, self.s13), (self.w2, self.s2) = q(2 * I, H, seed + 1), q(H, I, seed + 2)
        self.R = P + n_shared * T
        xc, xs = ref.encode(self.x)
        self.xq, self.xs = ref.pack(xc), xs

    @staticmethod
    def _weights(rows, cols, seed):
        c, s = ref.encode(rnd(rows, cols, seed=seed, scale=cols ** -0.5))
        return ref.pack(c), s

    def gpu(self):
        d = lambda t, dt=None: (t if dt is None else t.view(dt)).to(DEV)  # noqa: E731
        return dict(xq=d(self.xq, Q4), x_scale=d(self.xs, S8), expert_offsets=d(self.offsets),
                    permuted_pair=d(self.pair), w13=d(self.w13, Q4), w2=d(self.w2, Q4), w13_scale=d(self.s13, S8),
                    w2_scale=d(self.s2, S8), k=self.k, E=self.E, n_shared=self.sh)

    def rows_of(self, g):
        a, b = int(self.offsets[g]), int(self.offsets[g + 1])
        tok = self.pair[a:b].long() // self.k if g < self.E else torch.arange(self.T)
        return a, b, tok

    def check(self, got, ws):
        R, I = self.R, self.I
        ws = ws.cpu()
        hq = ws[:R * I // 2].view(R, I // 2)
        at = (R * I // 2 + 255) // 256 * 256
        hs = ws[at:at + R * I // 32].view(R, I // 32)
        x = ref.decode(self.xq, self.xs)
        got = got.cpu()
        for g in range(self.E + self.sh):
            a, b, tok = self.rows_of(g)
            if a == b:
                continue
            h, off = ref.h_of(x[tok], ref.decode(self.w13[g], self.s13[g]))
            ok = ref.may_be(hq[a:b], hs[a:b], h, off)
            assert bool(ok.all()), f"group {g}: {int((~ok).sum())} of {ok.numel()} codes of h are of other values"
            want, err = ref.out_of(ref.decode(hq[a:b], hs[a:b]), ref.decode(self.w2[g], self.s2[g]))
            within(got[a:b], want, want.abs() * half_step(BF) * (1 + 2 ** -7) + err + 1e-38, f"rows of group {g}")


def run(case, **kw):
    ws = torch.full((moe.binding.workspace_size(case.T, case.k, case.E, case.sh, case.H, case.I, Q4),), 0xA5, dtype=U8,
                    device=DEV)
    out = Guarded()
    rows = out((case.R, case.H), BF)
    got = moe.expert_ffn_mxfp4(**case.gpu(), ws=ws, out=rows, **kw)
    assert got is rows
    out.check()
    return rows, ws


@pytest.mark.parametrize("H,I", [(128, 128), (256, 128), (384, 640), (1024, 256), (640, 384)])
@pytest.mark.parametrize("counts", [(1,), (5, 0, 70, 31), (33, 1, 400)])
def test_ffn(counts, H, I):
    c = Case(counts, H, I)
    c.check(*run(c))


@pytest.mark.parametrize("H,I", [(2560, 2688), (1792, 2304), (1408, 1536)])
def test_ffn_long_rows(H, I):
    """Rings that go round, in each class of tiles: 5.5 to 10.5 stages, scales in one transfer and in four."""
    case = Case((33, 1, 400, 90), H, I)
    case.check(*run(case))


def test_ffn_shared_and_several_places():
    c = Case((40, 0, 12, 8), 256, 256, n_shared=2, k=3, seed=5)
    c.check(*run(c))


@pytest.mark.parametrize("n", [63, 64, 65, 127, 128, 129, 255, 256, 383, 384, 385, 511, 513, 641])
def test_ffn_class_borders(n):
    """Row counts on both sides of every tile and class border."""
    c = Case((n, 2, n + 1), 256, 128, seed=n)
    c.check(*run(c))


@pytest.mark.parametrize("H,I", [(128, 2048), (4096, 128)])
def test_ffn_many_rows(H, I):
    """Enough of them that groups past 128 rows take the largest tiles, in FC1 and in FC2."""
    case = Case((64, 128, 129, 200, 256, 257, 300, 383, 384, 700, 33, 5400), H, I)
    case.check(*run(case))


@pytest.mark.parametrize("H,I,E", [(256, 256, 256), (4096, 1152, 40), (1152, 4096, 70), (2688, 1408, 40)])
def test_ffn_classes(H, I, E):
    """Every class of tiles, its borders and the rows it hands on, in a call of more tiles than one
    round of the chip (which has them all alike)."""
    counts = [63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 400, 513, 640, 1, 2, 31]
    counts = np.random.default_rng(E).permutation(counts + [0] * (E - len(counts))).tolist()
    case = Case(counts, H, I, alike=True)
    case.check(*run(case))


@pytest.mark.parametrize("n", [400, 513, 640])
def test_ffn_hand_off(n):
    """Long rows: a big group's remainder goes to the smaller tiles, in FC1 and in FC2."""
    for H, I in ((4096, 128), (256, 4224)):
        c = Case((n, 3), H, I, seed=n)
        c.check(*run(c))


def test_ffn_of_the_layer_calls():
    """quantise, route, permute, FFN, finalize as a layer runs them, against 64 bits on the same codes."""
    T, H, I, E, k, sh = 75, 512, 256, 16, 4, 1
    x, logits = rnd(T, H, dt=BF), rnd(T, E, seed=3)
    G = E + sh
    w13, w2 = rnd(G * 2 * I, H, seed=1, scale=H ** -0.5).to(DEV), rnd(G * H, I, seed=2, scale=I ** -0.5).to(DEV)
    q13, s13 = moe.quantize_mxfp4(w13)
    q2, s2 = moe.quantize_mxfp4(w2)
    q13, s13, q2, s2 = q13.view(G, 2 * I, -1), s13.view(G, 2 * I, -1), q2.view(G, H, -1), s2.view(G, H, -1)
    ids, scales = moe.route(logits.to(DEV), k, moe.ROUTE_RENORMALIZE)
    off, pair, up = moe.permute(ids, E, sh)
    xq, xs = moe.quantize_mxfp4(x.to(DEV))
    rows = moe.expert_ffn_mxfp4(xq, xs, off, pair, q13, q2, s13, s2, k, E, sh)
    got = moe.finalize(rows, up, scales, sh).cpu()
    x64, want = ref.near(x), torch.zeros(T, H, dtype=F64)
    d13, d2 = ref.decode(to_bytes(q13), to_bytes(s13)), ref.decode(to_bytes(q2), to_bytes(s2))
    ids, scales = ids.cpu(), scales.cpu().to(F64)

    def expert(e, v):
        h, _ = ref.h_of(v, d13[e])
        return ref.near(h) @ d2[e].t()

    for t in range(T):
        for j in range(k):
            want[t] += scales[t, j] * expert(int(ids[t, j]), x64[t:t + 1])[0]
    want += expert(E, x64)
    far = float((got.to(F64) - want).norm() / want.norm())
    # two bf16 roundings, each 2^-8 at most; a code of h on the other side of its border is rare
    assert far < 2 * half_step(BF), far


def test_ffn_nan_stays_in_its_rows():
    c = Case((20, 300), 256, 256, seed=9)
    clean, _ = run(c)
    c.xs[7, 3] = 255
    got, _ = run(c)
    hit = torch.zeros(c.R, dtype=torch.bool)
    for g in range(2):
        a, b, tok = c.rows_of(g)
        hit[a:b] = tok == 7
    assert bool(got.cpu()[hit].isnan().all()) and torch.equal(bits(got)[~hit], bits(clean)[~hit])
    c.xs[7, 3] = 127
    c.s2[1, 5, 2] = 255
    got, _ = run(c)
    assert bool(got.cpu()[20:, 5].isnan().all())
    rest = [i for i in range(256) if i != 5]
    assert not bool(got.cpu()[:, rest].isnan().any()) and not bool(got.cpu()[:20].isnan().any())


def test_ffn_extreme_scales():
    """Scales at both ends: products past fp32's range are infinite or zero, and none of it is a NaN
    where 64 bits have none."""
    c = Case((40,), 256, 128)
    c.xs[:] = 0
    c.s13[:] = 10
    got, _ = run(c)
    assert bool((got == 0).all())  # gates below the smallest number
    c = Case((40,), 256, 128)
    c.s2[:] += 60
    c.check(*run(c))


def test_ffn_repeats_and_side_stream_and_graphs():
    cases = [Case((50, 7, 210), 512, 256, seed=s) for s in (1, 2)]
    eager = [run(c)[0].clone() for c in cases]
    for c, e in zip(cases, eager):
        same(run(c)[0], e, "again")
    ins = [c.gpu() for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.expert_ffn_mxfp4(**ins[0])
    side.synchronize()
    same(got, eager[0], "side stream")
    c = cases[0]
    ws = moe.alloc_workspace(c.T, c.k, c.E, c.sh, c.H, c.I, Q4)
    x = [rnd(c.T, c.H, seed=70 + i, dt=BF).to(DEV) for i in range(2)]

    def step(i):
        q, s = moe.quantize_mxfp4(x[i])
        v = moe.dequantize_mxfp4(q, s)
        return v, moe.expert_ffn_mxfp4(**dict(ins[i], xq=q, x_scale=s), ws=ws)

    want = [[t.clone() for t in step(i)] for i in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step(i)))
    for turn in range(4):
        for i, (g, out) in enumerate(graphs):
            for t in out:
                t.view(U8).fill_(0x5A)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want[i]):
                same(a, b, f"graph {i}, replay {turn}")
            step(1 - i)


def test_ffn_row_does_not_depend_on_the_batch():
    """A row's result is the same alone and among others of its tile class."""
    c = Case((30,), 512, 256)
    whole, _ = run(c)
    one = c.gpu()
    row = 17
    tok = int(c.pair[row])
    one.update(xq=one["xq"].view(U8)[tok:tok + 1].clone().view(Q4), x_scale=one["x_scale"].view(U8)[tok:tok + 1].clone().view(S8),
               expert_offsets=torch.tensor([0, 1], dtype=torch.int32, device=DEV),
               permuted_pair=torch.zeros(1, dtype=torch.int32, device=DEV))
    same(moe.expert_ffn_mxfp4(**one)[0], whole[row], "row")


def test_ffn_past_32_bits():
    """Rows of fc2_out past 2^32 bytes, 256 experts: a late row equals the same row in a small call."""
    T, H, I, E, k = 40_000, 7168, 128, 256, 8
    g = torch.Generator(device=DEV).manual_seed(0)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=U8)  # noqa: E731
    near1 = lambda *s: torch.randint(118, 124, s, generator=g, device=DEV, dtype=U8)  # noqa: E731
    xq, xs = byte(T, H // 2), near1(T, H // 32)
    w13, s13, w2, s2 = byte(E, 2 * I, H // 2), near1(E, 2 * I, H // 32), byte(E, H, I // 2), near1(E, H, I // 32)
    ids = torch.randn((T, E), generator=g, device=DEV).topk(k, 1).indices.int()
    off, pair, up = moe.permute(ids, E)
    args = (w13.view(Q4), w2.view(Q4), s13.view(S8), s2.view(S8), k, E)
    rows = moe.expert_ffn_mxfp4(xq.view(Q4), xs.view(S8), off, pair, *args)
    assert rows.numel() * 2 > 1 << 32
    few = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV)
    o2, p2, u2 = moe.permute(ids[few].contiguous(), E)
    part = moe.expert_ffn_mxfp4(xq[few].contiguous().view(Q4), xs[few].contiguous().view(S8), o2, p2, *args)
    a = rows[up.view(T, k)[few].reshape(-1).long()].float()
    b = part[u2.long()].float()
    # the tile class sets the order of no sum: K steps go in order in every one
    assert torch.equal(a, b)


def test_ffn_refusals():
    c = Case((8, 8), 256, 128)
    good = c.gpu()
    moe.expert_ffn_mxfp4(**good)
    for name, bad in (("xq", good["xq"].view(U8)), ("x_scale", good["x_scale"].view(U8)),
                      ("w13", good["w13"].view(U8)), ("w13", good["w13"][0]), ("w13", good["w13"][:1]),
                      ("w2", good["w2"][:, :128]), ("w13_scale", good["w13_scale"][:, :, :4]),
                      ("w2_scale", good["w2_scale"][:1]), ("expert_offsets", good["expert_offsets"][:2]),
                      ("permuted_pair", good["permuted_pair"][:3])):
        with pytest.raises(ValueError):
            moe.expert_ffn_mxfp4(**{**good, name: bad})
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.expert_ffn_mxfp4(**good, ws=torch.empty(64, dtype=U8, device=DEV))
    with pytest.raises(ValueError):
        moe.expert_ffn_mxfp4(**good, out=torch.empty((16, 256), device=DEV))


def test_timing_names():
    x = rnd(8, 64).to(DEV)
    binding.timing_enable(True)
    try:
        binding.kernel_times(reset=True)
        moe.dequantize_mxfp4(*moe.quantize_mxfp4(x))
        t = binding.kernel_times(reset=True)
    finally:
        binding.timing_enable(False)
    for n in ("quantize_mxfp4", "dequantize_mxfp4"):
        assert t[n][1] == 1 and t[n][0] > 0
