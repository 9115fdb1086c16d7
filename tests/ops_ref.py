"""Plain 64-bit implementations of the router, the rows to their experts and back, and
the adapters, and the error bounds that their tests hold the kernels to."""

from __future__ import annotations

import numpy as np
import torch

# half a step relative to the value: the most one rounding to the type is off
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the spacing of the type's subnormals
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
U32 = 2.0 ** -24


def assert_close(got, ref, sums_off, name=""):
    """got (rounded once to its type) against the 64-bit ref: within sums_off (the bound
    on the float32 sums' error, elementwise) plus half a step of the type at the value."""
    half, tiny = HALF[got.dtype], TINY[got.dtype]
    g = got.detach().cpu().double()
    ref, sums_off = ref.cpu().double(), sums_off.cpu().double()
    allowed = sums_off + half * (ref.abs() + sums_off) + tiny
    bad = ~((g - ref).abs() <= allowed)
    bad &= ~((g == ref) | (g.isnan() & ref.isnan()))       # infinities and NaN alike
    n = int(bad.sum())
    if n:
        at = tuple(int(i[0]) for i in torch.nonzero(bad, as_tuple=True))
        raise AssertionError("%s: %d of %d off, first at %s: %r against %r, allowed %.3g" % (
            name, n, g.numel(), at, float(g[at]), float(ref[at]), float(allowed[at])))


# ---- router ---------------------------------------------------------------------------

def route(logits, K, renorm):
    """ids int32 [T, K], weights float64 [T, K], the softmax p [T, E] they come from, and
    the largest |l - m| of each token."""
    l = logits.cpu().double().numpy()
    T, E = l.shape
    ids = np.full((T, K), -1, np.int32)
    w = np.zeros((T, K))
    p = np.zeros((T, E))
    reach = np.zeros(T)
    for t in range(T):
        ok = [e for e in range(E) if l[t, e] > -np.inf]
        order = sorted(ok, key=lambda e: (-l[t, e], e))[:K]
        if not order:
            continue
        m = l[t, order[0]]
        over = order if renorm else ok
        with np.errstate(invalid="ignore"):
            d = np.array([0.0 if l[t, e] == m else l[t, e] - m for e in over])
        ex = np.exp(d)
        reach[t] = np.abs(d[np.isfinite(d)]).max(initial=0.0)
        p[t, over] = ex / ex.sum()
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
    return ids, torch.from_numpy(w), torch.from_numpy(p), torch.from_numpy(reach)


def route_backward(ids, w, p, dw, E, renorm):
    """dlogits float64 [T, E] and the magnitudes |p| (|g| + sum |w g|) its error goes by."""
    ids, w, dw = ids.cpu().long(), w.cpu().double(), dw.cpu().double()
    T, K = ids.shape
    dl, mag = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        g = torch.zeros(E, dtype=torch.float64)
        pt = p[t].clone()
        if renorm:
            pt.zero_()
        dot, size = 0.0, 0.0
        for k in range(K):
            e = int(ids[t, k])
            if 0 <= e < E:
                g[e] += dw[t, k]
                if renorm:
                    pt[e] = w[t, k]
                dot += float(w[t, k] * dw[t, k])
                size += abs(float(w[t, k] * dw[t, k]))
        dl[t] = pt * (g - dot)
        mag[t] = pt * (g.abs() + size)
    return dl, mag


# ---- rows -----------------------------------------------------------------------------

def route_rows(route_row, T, K, R):
    """(slot, row) of the slots that name a row."""
    rr = route_row.cpu().long().reshape(-1)[:T * K]
    slot = torch.nonzero((rr >= 0) & (rr < R))[:, 0]
    return slot, rr[slot]


def unpermute(rows, w, route_row, T, K):
    """out float64 [T, H] and the sum of its terms' magnitudes."""
    y = rows.cpu().double()
    slot, row = route_rows(route_row, T, K, y.shape[0])
    terms = y[row]
    if w is not None:
        terms = terms * w.cpu().double().reshape(-1)[slot][:, None]
    out = torch.zeros(T, y.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    tok = torch.div(slot, K, rounding_mode="floor")
    out.index_add_(0, tok, terms)
    mag.index_add_(0, tok, terms.abs())
    return out, mag


# ---- adapters -------------------------------------------------------------------------

def adapters(x, w, base, ids, a, b, scale):
    """out float64 [T, N], and the bound on the float32 sums' error: H terms of x W^T and of
    x A^T, rank terms of v B^T, each sum of n terms off by at most (n + 2) 2^-24 of the
    terms' magnitudes; v enters as hi + lo, off by at most 2^-17 of its row's largest."""
    x64 = x.cpu().double()
    T, H = x64.shape
    a, b, ids = a.cpu().double(), b.cpu().double(), ids.cpu().long()
    L, r = a.shape[0], a.shape[1]
    if w is not None:
        w64 = w.cpu().double()
        out = x64 @ w64.t()
        off = (H + 2) * U32 * (x64.abs() @ w64.abs().t())
    else:
        out = base.cpu().double().clone()
        off = 2 * U32 * out.abs()
    for l in range(L):
        at = torch.nonzero(ids == l)[:, 0]
        if not at.numel():
            continue
        s = 1.0 if scale is None else float(scale[l])
        v = x64[at] @ a[l].t()
        vm = x64[at].abs() @ a[l].abs().t()
        out[at] += s * (v @ b[l].t())
        v_off = (H + 2) * U32 * vm + 2.0 ** -17 * v.abs().amax(1, keepdim=True)
        off[at] += abs(s) * (v_off @ b[l].abs().t()
                             + (r + 6) * U32 * ((v.abs() + v_off) @ b[l].abs().t()))
    return out, off + 2 * U32 * (out.abs() + off)
