"""Plain 64-bit forms of the row operators (norm, dispatch, activation, and
the gradients), on the CPU, written from the formulas.  Nothing here calls the
library.  Where a formula differentiates, `differences` checks it."""
from __future__ import annotations

import torch

F64 = torch.float64
EPS32 = 2.0 ** -24  # half a step of fp32


def half_step(dt) -> float:
    return torch.finfo(dt).eps / 2


def rmsnorm(z, w, eps):
    z, w = z.to(F64), w.to(F64)
    return z * w / (z.square().mean(1, keepdim=True) + eps).sqrt()


def rmsnorm_backward(dy, z, w, eps, dsum=None):
    """(dz, dweight, and for each a bound on the size of the terms it sums)."""
    dy, z, w = dy.to(F64), z.to(F64), w.to(F64)
    H = z.shape[1]
    c = (z.square().mean(1, keepdim=True) + eps).rsqrt()
    g = dy * w
    dz = c * g - z * c ** 3 * (g * z).sum(1, keepdim=True) / H
    size = (c * g).abs() + (z * c ** 3).abs() * (g * z).abs().sum(1, keepdim=True) / H
    if dsum is not None:
        dz = dz + dsum.to(F64)
        size = size + dsum.to(F64).abs()
    terms = dy * z * c
    return dz, terms.sum(0), size, terms.abs().sum(0)


def dispatch(x, unpermute, k, n_shared):
    T = x.shape[0]
    rows = torch.zeros((T * (k + n_shared),) + x.shape[1:], dtype=x.dtype)
    for t in range(T):
        for j in range(k):
            rows[unpermute[t * k + j]] = x[t]
        for s in range(n_shared):
            rows[T * k + s * T + t] = x[t]
    return rows


def dispatch_backward(d_rows, unpermute, k, n_shared):
    """(dx, the sum of its terms' sizes); a pair outside [0, T*k) adds nothing."""
    T = unpermute.numel() // k
    d = d_rows.to(F64)
    dx, size = torch.zeros((T, d.shape[1]), dtype=F64), torch.zeros((T, d.shape[1]), dtype=F64)
    for t in range(T):
        at = [int(r) for r in unpermute[t * k:(t + 1) * k] if 0 <= r < T * k]
        for r in at + [T * k + s * T + t for s in range(n_shared)]:
            dx[t] += d[r]
            size[t] += d[r].abs()
    return dx, size


def finalize(fc2, unpermute, scales, n_shared):
    T, k = scales.shape
    f, y = fc2.to(F64), torch.zeros((T, fc2.shape[1]), dtype=F64)
    for j in range(k):
        y += scales[:, j:j + 1].to(F64) * f[unpermute.view(T, k)[:, j].long()]
    for s in range(n_shared):
        y += f[T * k + s * T:T * k + (s + 1) * T]
    return y


def route_scales(logits, ids, method, scaling, renorm):
    """moe_route's weights of the given experts."""
    l = logits.to(F64)
    kept = l.gather(1, ids.long())
    if method == 0 and not renorm:
        return scaling * torch.softmax(l, 1).gather(1, ids.long())
    if method in (0, 1, 4):
        return scaling * torch.softmax(kept, 1)
    sig = torch.sigmoid(kept)
    if method == 3:
        return scaling * sig
    return scaling * sig / (sig.sum(1, keepdim=True) + (1e-20 if method == 2 else 0.0))


def route_backward(logits, ids, d_scales, method, scaling, renorm):
    """(d_logits, the size of the terms of each)."""
    l, i = logits.to(F64), ids.long()
    T, E = l.shape
    v = scaling * d_scales.to(F64)
    kept = l.gather(1, i)
    zero = torch.zeros((T, E), dtype=F64)
    if method == 0 and not renorm:
        p = torch.softmax(l, 1)
        pk = p.gather(1, i)
        mean, size = (v * pk).sum(1, keepdim=True), (v * pk).abs().sum(1, keepdim=True)
        return (p * (zero.scatter_add(1, i, v) - mean),
                p * (zero.scatter_add(1, i, v.abs()) + size))
    if method in (0, 1, 4):
        q = torch.softmax(kept, 1)
        d, s = q * (v - (v * q).sum(1, keepdim=True)), q * (v.abs() + (v * q).abs().sum(1, keepdim=True))
    else:
        sig = torch.sigmoid(kept)
        slope = sig * torch.sigmoid(-kept)
        if method == 3:
            d, s = v * slope, (v * slope).abs()
        else:
            S = sig.sum(1, keepdim=True) + (1e-20 if method == 2 else 0.0)
            d = slope / S * (v - (v * sig / S).sum(1, keepdim=True))
            s = slope / S * (v.abs() + (v * sig / S).abs().sum(1, keepdim=True))
    return zero.scatter_add(1, i, d), zero.scatter_add(1, i, s)


def swiglu(gu):
    I = gu.shape[1] // 2
    g, u = gu[:, :I].to(F64), gu[:, I:].to(F64)
    return g * torch.sigmoid(g) * u


def swiglu_backward(dh, gu):
    """(d_gu, the size of its terms)."""
    I = gu.shape[1] // 2
    g, u, d = gu[:, :I].to(F64), gu[:, I:].to(F64), dh.to(F64)
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    dg, du = d * u * s * (1 + g * r), d * g * s
    return torch.cat([dg, du], 1), torch.cat([(d * u * s).abs() * (1 + (g * r).abs()), du.abs()], 1)


def values(codes, scales):
    """code * scale of 1x128 e4m3 blocks."""
    rows, cols = codes.shape
    return (codes.float().to(F64).view(rows, cols // 128, 128) * scales.to(F64)[:, :, None]).view(rows, cols)


def code_tolerance(v, scales):
    """How far an e4m3 code's value may be from v: half a step, 2^-4 of the value for normal codes
    and 2^-10 of the scale below."""
    rows, cols = v.shape
    s = scales.to(F64)[:, :, None].expand(rows, cols // 128, 128).reshape(rows, cols)
    return torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10)


def differences(f, x, direction, step):
    """Slope of the number f(x) along `direction` by central differences."""
    return float((f(x + step * direction) - f(x - step * direction)) / (2 * step))
