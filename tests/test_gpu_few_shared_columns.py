"""The layer for few tokens where workgroups share columns of y (H up to 2048): at the I whose rows give
every wave of them as many pieces, y of a token is the token's own, whatever else is in the call.  That
holds bit for bit, so the weights need no 64-bit values here."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_07_amd as moe
import oracle
from test_gpu_few import Q4, RENORM, S8, U8, Layer
from test_gpu_rowops import BF, DEV, F8, FP, rnd, same

pytestmark = pytest.mark.gpu

# the I of one workgroup a column, times n = 8, 4, 2 and, past 2048, 1 of them
BASE = dict(f32=512, bf16=1024, fp8=1024, mxfp4=2048)
COLUMNS = [(128, 8), (512, 8), (640, 4), (1024, 4), (1152, 2), (2048, 2), (2176, 1)]


class Quick(Layer):
    """A Layer of random weights made on the GPU."""

    def __init__(self, T, H, I, E, k, wdt, n_shared=0, method=RENORM, seed=0):
        self.T, self.H, self.I, self.E, self.k, self.wdt, self.sh = T, H, I, E, k, wdt, n_shared
        self.dt = FP if wdt == "f32" else BF
        self.x, self.logits = rnd(T, H, seed=seed).to(self.dt), rnd(T, E, seed=seed + 1)
        self.method, self.routing = method, {}
        gen = torch.Generator(device=DEV).manual_seed(seed)
        (self.w13, self.s13), (self.w2, self.s2) = (self.matrices(gen, E + n_shared, N, K) for N, K in ((2 * I, H), (H, I)))

    def matrices(self, gen, G, N, K):
        if self.wdt == "mxfp4":
            codes = torch.randint(0, 256, (G, N, K // 2), generator=gen, device=DEV, dtype=U8)
            # codes of all sizes have a mean square of 2.93^2
            e = 127 - round(np.log2(2.93 * K ** 0.5))
            return codes.view(Q4), torch.randint(e - 1, e + 2, (G, N, K // 32), generator=gen, device=DEV, dtype=U8).view(S8)
        v = torch.randn((G, N, K), generator=gen, device=DEV)
        if self.wdt == "fp8":
            s = (0.5 + torch.rand((G, N // 128, K // 128), generator=gen, device=DEV)) / 64 * K ** -0.5
            return (v * 64).clamp(-448, 448).to(F8), s
        return (v * K ** -0.5).to(self.dt), None


@pytest.mark.parametrize("H,n", COLUMNS)
@pytest.mark.parametrize("wdt", sorted(BASE))
def test_a_token_is_its_own(wdt, H, n):
    """Alone, among others in another place, beside NaN and infinities, and beside a token with every
    expert masked."""
    T, E, k = 19, 5, 2
    a = Quick(T, H, n * BASE[wdt], E, k, wdt, 1, seed=n)
    (y, ids, scales), h = a.run()
    assert bool(y.isfinite().all()) and bool((y != 0).any(1).all())
    g = a.gpu()
    _, _, up = oracle.permute(ids.cpu().numpy(), E, 1)
    up = torch.from_numpy(np.asarray(up)).view(T, k)
    for t in (0, 7, 18):
        (y1, i1, s1), h1 = a.run(x=g["x"][t:t + 1].clone(), logits=g["logits"][t:t + 1].clone())
        same(i1[0], ids[t], "ids")
        same(s1[0], scales[t], "scales")
        same(h1[:k], h[up[t][ids[t].cpu().argsort()].long().to(DEV)], "h")
        same(h1[k], h[T * k + t], "shared h")
        same(y1[0], y[t], "y")
    order = torch.from_numpy(np.random.default_rng(n).permutation(T)).to(DEV)
    (y2, _, _), _ = a.run(x=g["x"][order].contiguous(), logits=g["logits"][order].contiguous())
    same(y2, y[order], "y in another order")
    some = order[:9].sort().values
    (y2, _, _), _ = a.run(x=g["x"][some].contiguous(), logits=g["logits"][some].contiguous())
    same(y2, y[some], "y of some")
    x, l = g["x"].clone(), g["logits"].clone()
    x[5, 17], x[6, 3], l[2], l[11] = float("nan"), float("inf"), float("nan"), float("-inf")
    (y2, i2, _), _ = a.run(x=x, logits=l)
    rest = [t for t in range(T) if t not in (2, 5, 6, 11)]
    same(i2[rest], ids[rest], "ids")
    same(y2[rest], y[rest], "y beside other tokens' NaN")
    assert bool(y2[5].isnan().all()) and not bool(y2[6].isfinite().all())
    assert bool(((i2 >= 0) & (i2 < E)).all())
