"""Plain 64-bit implementations of the dense feed-forward block and of the residual joint,
with their gradients, and the error bounds that their tests hold the kernels to."""

from __future__ import annotations

import torch

from ops_ref import HALF, TINY, U32

# the hardware's exp, reciprocal and the products around them: 1 + exp(-g) is off by
# |g| 2^-24 (the rounded argument) and 2 ulps, each other step by at most 2
ACT = 12


def d(t):
    return t.detach().double()


def silu(g):
    return g / (1.0 + torch.exp(-g))


def cut(v, top):
    return torch.minimum(torch.maximum(v, torch.full_like(v, -top)), torch.full_like(v, top))


def below(v, top):
    return torch.minimum(v, torch.full_like(v, top))


def ffn_forward(x, w13, w2, gl, ul, base=None):
    """out, its bound, and g | u with theirs (all float64)."""
    half, tiny = HALF[x.dtype], TINY[x.dtype]
    x, w13, w2 = d(x), d(w13), d(w2)
    H, I = x.shape[1], w2.shape[1]
    gu = x @ w13.t()
    gu_off = (H + 2) * U32 * (x.abs() @ w13.abs().t())
    g, u = below(gu[:, :I], gl), cut(gu[:, I:], ul)
    h = silu(g) * u
    h_off = 1.1 * gu_off[:, :I] * (u.abs() + gu_off[:, I:]) + silu(g).abs() * gu_off[:, I:]
    h_off = h_off + (ACT + g.abs()) * U32 * (h.abs() + h_off)
    h_off = h_off + half * (h.abs() + h_off) + tiny
    out = h @ w2.t()
    off = h_off @ w2.abs().t() + (I + 2) * U32 * ((h.abs() + h_off) @ w2.abs().t())
    if base is not None:
        out = out + d(base)
        off = off + U32 * (out.abs() + off)
    return out, off, gu, gu_off


def mx_values(codes, scale):
    """The float64 values of MX FP8 rows [T, N] with exponent bytes [T, N/32]."""
    v = codes.view(torch.uint8).cpu().view(torch.float8_e4m3fn).double()
    e = scale.cpu().double() - 127
    return (v.reshape(v.shape[0], -1, 32) * torch.exp2(e)[:, :, None]).reshape(v.shape)


def mx_rows(v):
    """codes and exponent bytes of float64 rows, by the layer's 1x32 rule."""
    b = v.double().cpu().reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, 0).clamp(-127, 127)
    a = (b * torch.exp2(-e.double())).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.where(amax > 0, torch.round(a / step) * step, 0.0)
    codes = q.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(v.shape), (e[:, :, 0] + 127).to(torch.uint8)


def ffn_backward(dout, x, w13, w2, gu, gl, ul, dt):
    """dx, dw13, dw2 in float64 and their bounds; x and gu: the values that were kept; dt:
    the type that dg, du and h are rounded to."""
    half, tiny = HALF[dt], TINY[dt]
    dout, x, w13, w2, gu = d(dout), d(x), d(w13), d(w2), d(gu)
    T, H, I = x.shape[0], x.shape[1], w2.shape[1]
    g, u = below(gu[:, :I], gl), cut(gu[:, I:], ul)
    s = 1.0 / (1.0 + torch.exp(-g))
    dh = dout @ w2
    dh_off = (H + 2) * U32 * (dout.abs() @ w2.abs())
    slope = s * (1.0 + g * (1.0 - s))
    # 1 - s loses what s has in ulps of 1, so the slope's error is in those of 1 + |g|
    slope_off = (ACT + g.abs()) * U32 * (1.0 + g.abs())
    keep_g, keep_u = gu[:, :I] <= gl, gu[:, I:].abs() <= ul
    dg = torch.where(keep_g, dh * u * slope, 0.0)
    du = torch.where(keep_u, dh * g * s, 0.0)
    dg_off = (dh_off * (slope.abs() + slope_off) + dh.abs() * slope_off) * u.abs()
    du_off = dh_off * (g * s).abs() + (ACT + g.abs()) * U32 * (dh.abs() + dh_off) * (g * s).abs()
    q = torch.cat([dg, du], 1)
    q_off = torch.cat([dg_off, du_off], 1) + 4 * U32 * q.abs()
    q_off = torch.where(torch.cat([keep_g, keep_u], 1), q_off + half * (q.abs() + q_off) + tiny,
                        0.0)
    h = g * s * u
    h_off = (ACT + g.abs()) * U32 * h.abs()
    h_off = h_off + half * (h.abs() + h_off) + tiny

    def product(a, a_off, b, n):
        return a @ b, a_off @ b.abs() + (n + 2) * U32 * ((a.abs() + a_off) @ b.abs())

    dx, dx_off = product(q, q_off, w13, 2 * I)
    dw13, dw13_off = product(q.t(), q_off.t(), x, T)
    dw2, dw2_off = product(dout.t(), torch.zeros_like(dout).t(), h, T)
    dw2_off = dw2_off + (1 + (T + 2) * U32) * (dout.abs().t() @ h_off)
    return dx, dx_off, dw13, dw13_off, dw2, dw2_off


# ---- the joint ------------------------------------------------------------------------


def rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def norm_forward(x, w_pre, eps, skip, scale, y=None, w_post=None, gate=None):
    """res and its bound; res is what normed is the norm of, once rounded."""
    H = x.shape[1]
    r = d(x)
    if y is None:
        return r, torch.zeros_like(r)
    z = d(y)
    if w_post is not None:
        z = z * rms(z, eps) * d(w_post)
    a = scale * (torch.sigmoid(d(gate))[:, None] if gate is not None else 1.0)
    # the mean of H squares, its root, the gate and four products
    off = (H + 40) * U32 * (a * z).abs() + 4 * U32 * (skip * r).abs()
    return skip * r + a * z, off


def norm_of(stored, w_pre, eps):
    r = d(stored)
    n = r * rms(r, eps) * d(w_pre)
    return n, (r.shape[1] + 16) * U32 * n.abs()


def norm_backward(dnormed, dres, res, w_pre, eps, skip, scale, y=None, w_post=None, gate=None):
    """dict of (gradient, bound) in float64: dx, dw_pre, dy, dw_post, dgate."""
    some = dnormed if dnormed is not None else dres
    T, H = some.shape
    u = (H + 40) * U32
    dr = torch.zeros(T, H, dtype=torch.float64, device=some.device)
    size = torch.zeros_like(dr)
    if dres is not None:
        dr = dr + d(dres)
        size = size + d(dres).abs()
    out = {}
    if dnormed is not None:
        r, g = d(res), d(dnormed) * d(w_pre)
        q = rms(r, eps)
        dr = dr + q * g - r * q ** 3 * (g * r).mean(1, keepdim=True)
        size = size + (q * g).abs() + r.abs() * q ** 3 * (g * r).abs().mean(1, keepdim=True)
        t = d(dnormed) * r * q
        out["dw_pre"] = t.sum(0), (T + H + 60) * U32 * t.abs().sum(0)
    dr_off = u * size
    f = skip if y is not None else 1.0
    out["dx"] = f * dr, abs(f) * (dr_off + 2 * U32 * dr.abs())
    if y is None:
        return out
    s = torch.sigmoid(d(gate))[:, None] if gate is not None else torch.ones(
        T, 1, dtype=torch.float64, device=some.device)
    a, y = scale * s, d(y)
    dz, dz_off = a * dr, a.abs() * (dr_off + 40 * U32 * dr.abs())
    z = y
    if w_post is not None:
        w = d(w_post)
        q = rms(y, eps)
        z, g = y * q * w, dz * w
        t = dz * y * q
        out["dw_post"] = t.sum(0), ((T + H + 100) * U32 * t.abs() + dz_off * (y * q).abs()).sum(0)
        back = y.abs() * q ** 3
        out["dy"] = (q * g - y * q ** 3 * (g * y).mean(1, keepdim=True),
                     u * (q * g.abs() + back * (g * y).abs().mean(1, keepdim=True))
                     + q * dz_off * w.abs()
                     + back * (dz_off * (w * y).abs()).mean(1, keepdim=True))
    else:
        out["dy"] = dz, dz_off
    if gate is not None:
        k = (scale * s * (1.0 - s))[:, 0]
        m = (dr.abs() * z.abs()).sum(1)
        # sigmoid and 1 - sigmoid: the latter is off by ulps of 1
        k_off = abs(scale) * (40 * U32 * s * (1.0 - s) + 4 * U32 * s)[:, 0]
        out["dgate"] = (k * (dr * z).sum(1),
                        k.abs() * (2 * u * m + (dr_off * z.abs()).sum(1)) + k_off * m)
    return out
