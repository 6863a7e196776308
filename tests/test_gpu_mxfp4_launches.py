"""The 4-bit FFN in the launches that large calls take: a launch for each class of group sizes, where
the tiles are more than one round of the chip, and the largest tiles for groups past 128 rows, where
those are many.  Every case says how many launches each product has, so that a case cannot come to
test another path than the one it was written for; every expert has weights of its own."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_07_amd as moe
import mxfp4_ref as ref
from mixture_experts_layer_07_amd import binding
from rowops_ref import EPS32, half_step
from test_gpu_mxfp4 import Case, Guarded, Q4, U8
from test_gpu_rowops import BF, DEV, within

pytestmark = pytest.mark.gpu


class Coded(Case):
    """A Case whose weights are random codes (those of rounded normal values take minutes at these
    sizes), checked with the 64-bit products on the GPU."""

    @staticmethod
    def _weights(rows, cols, seed):
        gen = torch.Generator().manual_seed(seed)
        # codes of all sizes have a mean square of 2.93^2
        e = 127 - round(np.log2(2.93 * cols ** 0.5))
        return (torch.randint(0, 256, (rows, cols // 2), generator=gen, dtype=U8),
                torch.randint(e - 1, e + 2, (rows, cols // 32), generator=gen, dtype=U8))

    def run(self):
        """(rows, workspace, launches of FC1, launches of FC2)"""
        n = binding.workspace_size(self.T, self.k, self.E, self.sh, self.H, self.I, Q4)
        ws = torch.full((n,), 0xA5, dtype=U8, device=DEV)
        out = Guarded()
        rows = out((self.R, self.H), BF)
        binding.timing_enable(True)
        try:
            binding.kernel_times(reset=True)
            moe.expert_ffn_mxfp4(**self.gpu(), ws=ws, out=rows)
            t = binding.kernel_times(reset=True)
        finally:
            binding.timing_enable(False)
        out.check()
        return rows, ws, t["fc1"][1], t["fc2"][1]

    def check(self, got, ws):
        R, I = self.R, self.I
        ws = ws.cpu()
        hq = ws[:R * I // 2].view(R, I // 2)
        at = (R * I // 2 + 255) // 256 * 256
        hs = ws[at:at + R * I // 32].view(R, I // 32)
        x = ref.decode(self.xq, self.xs)
        got = got.cpu()
        seen = 0
        for g in range(self.E + self.sh):
            a, b, tok = self.rows_of(g)
            if a == b:
                continue
            h, off = ref.h_of(x[tok].to(DEV), ref.decode(self.w13[g], self.s13[g]).to(DEV))
            ok = ref.may_be(hq[a:b], hs[a:b], h.cpu(), off.cpu())
            assert bool(ok.all()), f"group {g}, {b - a} rows: {int((~ok).sum())} codes of h are of other values"
            want, err = ref.out_of(ref.decode(hq[a:b], hs[a:b]).to(DEV), ref.decode(self.w2[g], self.s2[g]).to(DEV))
            want, err = want.cpu(), err.cpu()
            within(got[a:b], want, want.abs() * half_step(BF) * (1 + 2 ** -7) + err + 1e-38, f"group {g}, {b - a} rows")
            seen += b - a
        assert seen == R

    def expect(self, fc1, fc2):
        rows, ws, n1, n2 = self.run()
        assert (n1, n2) == (fc1, fc2), "launches"
        self.check(rows, ws)


def scattered(counts, E, seed=0):
    """These group sizes among E experts, the rest without rows."""
    return np.random.default_rng([seed, E]).permutation(counts + [0] * (E - len(counts))).tolist()


BORDERS = [63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 400, 513, 640, 1, 2, 31]


@pytest.mark.parametrize("H,I,E", [(256, 256, 256), (640, 1408, 60), (2688, 1408, 24), (1152, 2176, 40)])
def test_classes(H, I, E):
    """Every class of tiles and its borders, rings that go round and half stages at their end."""
    Coded(scattered(BORDERS, E), H, I).expect(3, 3)


def test_classes_with_shared_experts():
    """Two places a token, two shared experts of more rows than any other."""
    c = Coded([90, 30, 0, 700, 130, 64, 200, 386], 2176, 1664, n_shared=2, k=2, seed=3)
    c.expect(3, 3)


@pytest.mark.parametrize("H,I", [(2560, 2688), (1792, 2304), (1408, 1664)])
def test_long_rows(H, I):
    """5.5 to 10.5 stages in each class, scales in one transfer and in four."""
    Coded(scattered([33, 1, 400, 90], 60), H, I).expect(3, 3)


@pytest.mark.parametrize("n", [384, 400, 512, 513, 640, 641])
@pytest.mark.parametrize("H,I", [(4096, 128), (256, 4224)])
def test_hand_off(n, H, I):
    """Long rows: a big group's remainder of up to 128 rows goes to the smaller tiles."""
    Coded(scattered([n, 3], 256, n), H, I, seed=n).expect(3, 3)


@pytest.mark.parametrize("n", [63, 64, 65, 127, 128, 129, 255, 256, 383, 384, 385, 511, 513, 641])
def test_class_borders(n):
    # no launch for a class that the call has too few rows for
    launches = 3 if 2 * n + 3 >= 384 else 2
    Coded(scattered([n, 2, n + 1], 256, n), 256, 128, seed=n).expect(launches, launches)


@pytest.mark.parametrize("n", [20, 31])
def test_no_class_past_the_first(n):
    """Fewer rows in the whole call than the second class has in a group: one launch, of the smallest tiles."""
    Coded([n, 0, 63 - n], 2304, 256).expect(1, 1)


MANY = [129, 255, 257, 383, 384, 385, 300, 200, 256, 130, 511, 513, 640, 63, 64, 128, 1, 0, 3593]


@pytest.mark.parametrize("H,I", [(4096, 4096), (4224, 4352)])
def test_large_tiles(H, I):
    """Groups of 129 rows and more on the largest tiles (more than 128 rows a group, and 512 such tiles
    and more in both products), many stages, remainders handed on (K of 4096 and more), a half stage at
    the end of the second shape's first product, and a shared expert."""
    assert sum(MANY) == 8192
    c = Coded(MANY, H, I, n_shared=1, k=2, seed=1)
    R, G = c.R, len(MANY) + 1
    assert R // G >= 128 and R // 256 * (H // 256) >= 512 and R // 256 * (2 * I // 256) >= 512
    c.expect(3, 3)


def test_large_tiles_short_rows():
    """The same without a hand-off (K below 4096), with one place a token."""
    c = Coded(MANY, 4096, 1024, seed=2)
    assert c.R // 256 * (2 * 1024 // 256) < 512  # FC1's groups past 128 rows take the middle tiles, FC2's the largest
    c.expect(3, 3)


def test_strongly_negative_gates():
    """Blocks of h whose gates are all far below zero: e^-g is off by 1.22 |g| half-steps of fp32 (its
    argument is rounded, and so is log2 e), so h is, relative to the block's own scale."""
    counts, H, I = (40, 90), 128, 128
    c = Case(counts, H, I, seed=4)
    rng = np.random.default_rng(7)
    pick = lambda v, *shape: torch.from_numpy(rng.choice(v, shape)).float()  # noqa: E731
    c.x[:, :16], c.x[:, 16:32] = 2.0, pick([-2.0, -1, -0.5, 0, 0.25, 1], c.T, 16)
    code, c.xs = ref.encode(c.x)
    c.xq = ref.pack(code)
    # Gates about -8, -24, -56 and -64, one of them for each block of h: eight weights a row that the
    # format has, and eight that vary them, on x's columns of 2.0
    w = torch.zeros(2, 2 * I, H)
    for g in range(2):
        for b, (size, n, unit) in enumerate(((0.5, 8, 0.125), (1.5, 8, 0.25), (4, 7, 1), (4, 8, 1))):
            rows = w[g, 32 * b:32 * b + 32]
            rows[:, :n] = -size
            rows[:, 8:16] = pick([-1.0, 0, 1], 32, 8) * unit
        w[g, I:] = torch.from_numpy(rng.standard_normal((I, H))).float()
    code, scale = ref.encode(w.view(-1, H))
    c.w13, c.s13 = ref.pack(code).view(2, 2 * I, -1), scale.view(2, 2 * I, -1)
    assert torch.equal(ref.decode(c.w13, c.s13)[:, :I].float(), w[:, :I])
    rows = torch.full((c.R, H), 0.0, dtype=BF, device=DEV)
    ws = torch.empty(binding.workspace_size(c.T, c.k, c.E, 0, H, I, Q4), dtype=U8, device=DEV)
    moe.expert_ffn_mxfp4(**c.gpu(), ws=ws, out=rows)
    host = ws.cpu()
    hq = host[:c.R * I // 2].view(c.R, -1)
    at = (c.R * I // 2 + 255) // 256 * 256
    hs = host[at:at + c.R * I // 32].view(c.R, -1)
    x = ref.decode(c.xq, c.xs)
    for g in range(2):
        a, b, tok = c.rows_of(g)
        d = ref.decode(c.w13[g], c.s13[g])
        gate, up = x[tok] @ d[:I].t(), x[tok] @ d[I:].t()
        assert bool((gate <= -6).all()) and float(gate.min()) < -66
        h = gate * torch.sigmoid(gate) * up
        # the gates are sums of few small multiples of a power of two: exact.  up has K/64 + 2 steps;
        # e^-g 1.22 |g|, and the exponential, 1 + e^-g, the reciprocal and two products 2 each
        size = x[tok].abs() @ d[I:].abs().t()
        off = h.abs() * EPS32 * (1.25 * gate.abs() + 12) + (gate * torch.sigmoid(gate)).abs() * EPS32 * (H / 64 + 2) * size
        ok = ref.may_be(hq[a:b], hs[a:b], h, off + 1e-45)
        assert bool(ok.all()), f"group {g}: {int((~ok).sum())} of {ok.numel()} codes of h are of other values"
