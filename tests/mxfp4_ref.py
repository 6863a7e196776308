"""Plain 64-bit forms of the 4-bit microscaled format and of the experts' FFN on it,
on the CPU, from the definitions.  Nothing here calls the library."""
from __future__ import annotations

import torch

from rowops_ref import EPS32, F64

LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64)
# the border above each code's values, the last open; a value on a border goes to the even code
BORDERS = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, torch.inf], dtype=F64)


def scale_bytes(amax):
    """Scale bytes of blocks with these largest magnitudes (64 bits); 255 where that is not finite."""
    finite = torch.isfinite(amax)
    e = torch.frexp(torch.where(finite, amax, torch.ones_like(amax))).exponent - 1 - 2 + 127
    e = torch.where(amax == 0, torch.zeros_like(e), e.clamp_min(0))
    return torch.where(finite, e, torch.full_like(e, 255))


def encode(v):
    """(codes uint8 [rows, cols], 0..15, scale bytes [rows, cols/32]) of v [rows, cols]; the codes of a
    block that is not finite are 0."""
    v = v.to(F64)
    rows, cols = v.shape
    b = v.view(rows, cols // 32, 32)
    s = scale_bytes(b.abs().amax(2).nan_to_num(nan=torch.inf))
    q = b.abs() * torch.exp2(127.0 - s.to(F64))[:, :, None]
    q = torch.where((s == 255)[:, :, None], torch.zeros_like(q), q)
    far = (q[..., None] - LEVELS).abs()
    # nearest level, the even code of two at the same distance: odd codes a little further off
    code = (far + 1e-12 * (torch.arange(8) % 2)).argmin(-1)
    sign = torch.signbit(b) & (s != 255)[:, :, None]
    return (code + 8 * sign).to(torch.uint8).view(rows, cols), s.to(torch.uint8)


def pack(codes):
    """Two codes a byte, the even column low."""
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).contiguous()


def unpack(packed):
    return torch.stack([packed % 16, packed // 16], -1).flatten(-2)


def decode(packed, scale):
    """The values of packed codes uint8 [.., cols/2] and scale bytes [.., cols/32], in 64 bits."""
    c = unpack(packed).long()
    v = LEVELS[c % 8] * torch.where(c >= 8, -1.0, 1.0)
    f = torch.where(scale == 255, torch.nan, torch.exp2(scale.to(F64) - 127))
    return (v.unflatten(-1, (-1, 32)) * f[..., None]).flatten(-2)


def near(v):
    """The values that v's codes stand for."""
    c, s = encode(v)
    return decode(pack(c), s)


def may_be(packed, scale, v, off):
    """Whether each code and scale may come from values within `off` of v."""
    rows, cols = v.shape
    lo, hi = (v.abs() - off).clamp_min(0), v.abs() + off
    top = lambda a: a.view(rows, cols // 32, 32).amax(2)  # noqa: E731
    s = scale.long()
    ok = (s >= scale_bytes(top(lo))) & (s <= scale_bytes(top(hi)))
    f = torch.exp2(s.to(F64) - 127).repeat_interleave(32, 1)
    c = unpack(packed).long()
    size = c % 8
    below = torch.where(size == 0, torch.zeros_like(lo), BORDERS[(size - 1).clamp_min(0)])
    inside = (hi >= below * f) & (lo <= BORDERS[size] * f)
    sign = (c >= 8) == torch.signbit(v)
    return ok.repeat_interleave(32, 1) & inside & (sign | (size == 0) | (v.abs() <= off))


def h_of(x, w13):
    """(h, how far fp32 work may put it off) of rows x and one expert's weights, all in 64 bits.
    A product sums K terms in K/64 steps, each of them half a step of fp32 of what has been summed;
    SwiGLU's exponential, reciprocal and products are within 8 half-steps together."""
    I = w13.shape[0] // 2
    gu, size = x @ w13.t(), x.abs() @ w13.abs().t()
    err = (x.shape[1] / 64 + 2) * EPS32 * size
    g, u = gu[:, :I], gu[:, I:]
    sig = torch.sigmoid(g)
    h = g * sig * u
    slope = (sig * (1 + g * (1 - sig))).abs()
    # the slope changes by at most 1/2 for each unit of the gate
    off = (u.abs() + err[:, I:]) * (slope + 0.5 * err[:, :I]) * err[:, :I] + (g * sig).abs() * err[:, I:]
    return h, off + 16 * EPS32 * h.abs() + 1e-37


def out_of(h, w2):
    """(rows, how far fp32 work may put them off) of given h."""
    return h @ w2.t(), (h.shape[1] / 64 + 2) * EPS32 * (h.abs() @ w2.abs().t())
