"""The residual joint with its norms on the GPU, against 64 bits inside derived bounds."""

import math

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ffn_ref
from ops_ref import assert_close

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(g, dt, T, H, std=1.0):
    return (torch.randn(T, H, generator=g, device=DEV) * std).to(dt)


SIZES = [(1, 32), (3, 96), (2, 160), (5, 512), (7, 544), (64, 1024), (130, 2080), (33, 2304),
         (600, 4096), (9, 5120), (300, 7168), (4, 8192), (3, 12320), (2, 16384)]


def _case(T, H, dt, seed, y=True, post=True, gated=True):
    g = _gen(seed)
    c = dict(x=_rows(g, dt, T, H), w_pre=1 + _rows(g, F32, 1, H, 0.2)[0])
    c["w_pre"] = c["w_pre"].to(dt)
    c["y"] = _rows(g, dt, T, H, 0.7) if y else None
    c["w_post"] = (1 + _rows(g, F32, 1, H, 0.2)[0]).to(dt) if y and post else None
    c["gate"] = torch.randn(T, generator=g, device=DEV) * 2 if y and gated else None
    c["dnormed"], c["dres"] = _rows(g, dt, T, H), _rows(g, dt, T, H)
    return c


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("T,H", SIZES)
def test_joint(T, H, dt):
    for y, post, gated in ((True, True, True), (True, False, True), (True, True, False),
                           (True, False, False), (False, False, False)):
        c = _case(T, H, dt, T * H + 2 * post + gated, y, post, gated)
        s = moe.NormShape(T=T, H=H, eps=1e-5, skip_scale=1.25, block_scale=0.4)
        what = "%s %s %s" % (y, post, gated)
        res = torch.full((T + 1, H), -3.0, dtype=dt, device=DEV) if y else None
        normed = torch.full((T + 1, H), -3.0, dtype=dt, device=DEV)
        moe.moe_norm_forward(s, c["x"], c["w_pre"], normed[:T], y=c["y"], w_post=c["w_post"],
                             gate=c["gate"], res=res[:T] if y else None)
        ref, off = ffn_ref.norm_forward(c["x"], None, 1e-5, 1.25, 0.4, c["y"], c["w_post"],
                                        c["gate"])
        stored = c["x"]
        if y:
            assert_close(res[:T], ref, off, "res " + what)
            assert (res[T] == -3).all()
            stored = res[:T].clone()
        n, n_off = ffn_ref.norm_of(stored, c["w_pre"], 1e-5)
        assert_close(normed[:T], n, n_off, "normed " + what)
        assert (normed[T] == -3).all()
        # the gradients, from what was stored
        o = dict(dx=torch.full((T + 1, H), -3.0, dtype=dt, device=DEV),
                 dw_pre=torch.empty(H, device=DEV))
        if y:
            o["dy"] = torch.full((T + 1, H), -3.0, dtype=dt, device=DEV)
        if post:
            o["dw_post"] = torch.empty(H, device=DEV)
        if gated:
            o["dgate"] = torch.empty(T, device=DEV)
        ws = moe.alloc_norm_workspace(s, DEV)
        cut = {k: v[:T] if v.shape[0] == T + 1 and v.dim() == 2 else v for k, v in o.items()}
        moe.moe_norm_backward(s, c["dnormed"], stored, c["w_pre"], cut["dx"], o["dw_pre"], ws,
                              dres=c["dres"], y=c["y"], w_post=c["w_post"], gate=c["gate"],
                              dy=cut.get("dy"), dw_post=o.get("dw_post"), dgate=o.get("dgate"))
        r = ffn_ref.norm_backward(c["dnormed"], c["dres"], stored, c["w_pre"], 1e-5, 1.25, 0.4,
                                  c["y"], c["w_post"], c["gate"])
        for k, (v, b) in r.items():
            assert_close(cut[k], v, b, "%s %s" % (k, what))
        for k in ("dx", "dy"):
            assert k not in o or (o[k][T] == -3).all()


@pytest.mark.parametrize("dt", [BF, F16, F32])
def test_parts_and_places(dt):
    """Without the norm behind, without dres, in place: the full call's bits."""
    T, H = 37, 1056
    c = _case(T, H, dt, 5)
    s = moe.NormShape(T=T, H=H, block_scale=0.5)
    ws = moe.alloc_norm_workspace(s, DEV)
    kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
    res, normed = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    moe.moe_norm_forward(s, c["x"], c["w_pre"], normed, res=res, **kw)
    only = torch.empty_like(res)
    moe.moe_norm_forward(s, c["x"], None, None, res=only, **kw)
    assert torch.equal(only, res)
    moe.moe_norm_forward(s, c["x"], c["w_pre"], only, **kw)            # res not stored
    assert torch.equal(only, normed)
    for into in ("x", "y"):
        v = {**c, into: c[into].clone()}
        moe.moe_norm_forward(s, v["x"], c["w_pre"], only, res=v[into], y=v["y"],
                             w_post=c["w_post"], gate=c["gate"])
        assert torch.equal(v[into], res) and torch.equal(only, normed)
    # the residual gradient alone
    dx, dy, dg = torch.empty_like(res), torch.empty_like(res), torch.empty(T, device=DEV)
    dwp, dwq = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    moe.moe_norm_backward(s, None, None, None, dx, None, ws, dres=c["dres"], dy=dy, dw_post=dwq,
                          dgate=dg, **kw)
    r = ffn_ref.norm_backward(None, c["dres"], None, None, 1e-6, 1.0, 0.5, **kw)
    for t, k in ((dx, "dx"), (dy, "dy"), (dwq, "dw_post"), (dg, "dgate")):
        assert_close(t, *r[k], k)
    # no dres
    moe.moe_norm_backward(s, c["dnormed"], res, c["w_pre"], dx, dwp, ws, dy=dy, dw_post=dwq,
                          dgate=dg, **kw)
    r = ffn_ref.norm_backward(c["dnormed"], None, res, c["w_pre"], 1e-6, 1.0, 0.5, **kw)
    for t, k in ((dx, "dx"), (dy, "dy"), (dwq, "dw_post"), (dg, "dgate"), (dwp, "dw_pre")):
        assert_close(t, *r[k], k)
    # in place
    full = [dx.clone(), dy.clone()]
    for into in ("dnormed", "res"):
        v = {**c, "res": res, into: (res if into == "res" else c[into]).clone(), "y": c["y"].clone()}
        moe.moe_norm_backward(s, v["dnormed"], v["res"], c["w_pre"], v[into], dwp, ws, y=v["y"],
                              w_post=c["w_post"], gate=c["gate"], dy=v["y"], dgate=dg)
        assert torch.equal(v[into], full[0]) and torch.equal(v["y"], full[1])
    v = dict(dres=c["dres"].clone())
    moe.moe_norm_backward(s, c["dnormed"], res, c["w_pre"], dx, dwp, ws, dres=c["dres"], **kw)
    moe.moe_norm_backward(s, c["dnormed"], res, c["w_pre"], v["dres"], None, None,
                          dres=v["dres"], **kw)
    assert torch.equal(v["dres"], dx)


@pytest.mark.parametrize("T,H", [(1, 128), (37, 7168), (200, 5120), (3, 16384), (5, 96)])
def test_mx_rows_are_the_quantisers(T, H):
    """normed as MX FP8: the bytes that moe_quant_mxfp8 makes of the bf16 normed; fp16 and
    float32 rows by the same rule."""
    for dt in (BF, F16, F32):
        c = _case(T, H, dt, T + H)
        s = moe.NormShape(T=T, H=H)
        normed = torch.empty_like(c["x"])
        codes = torch.full((T + 1, H), 99, dtype=torch.uint8, device=DEV)
        exps = torch.full((T + 1, H // 32), 99, dtype=torch.uint8, device=DEV)
        if T > 1:
            c["x"][0] = 0                                   # a row of nothing: all codes 0
            c["y"][0] = 0
        kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
        moe.moe_norm_forward(s, c["x"], c["w_pre"], normed, normed_fp8=codes[:T],
                             normed_scale=exps[:T], **kw)
        want, we = ffn_ref.mx_rows(normed)
        got = codes[:T].cpu()
        zero = (want & 0x7f) == 0
        assert torch.equal(exps[:T].cpu(), we), dt
        assert torch.equal(torch.where(zero, got & 0x7f, got), torch.where(zero, 0, want)), dt
        assert (codes[T] == 99).all() and (exps[T] == 99).all()
        alone, ae = torch.empty_like(codes[:T]), torch.empty_like(exps[:T])
        moe.moe_norm_forward(s, c["x"], c["w_pre"], None, normed_fp8=alone, normed_scale=ae, **kw)
        assert torch.equal(alone, codes[:T]) and torch.equal(ae, exps[:T])
        if dt == BF and H % 128 == 0:
            q = moe.MoeShape(T=T, H=H, I=128, K=1, E_total=1, E_local=1)
            qc, qs = torch.empty_like(alone), torch.empty_like(ae)
            moe.moe_quant_mxfp8(q, normed, qc, qs)
            assert torch.equal(qc, alone) and torch.equal(qs, ae)


def test_rows_of_nothing_and_of_nan():
    """Zeros with eps 0 and without, infinities and NaN: in their rows alone."""
    T, H = 6, 512
    c = _case(T, H, BF, 8)
    s = moe.NormShape(T=T, H=H)
    ws = moe.alloc_norm_workspace(s, DEV)
    out = torch.empty_like(c["x"])
    moe.moe_norm_forward(s, c["x"], c["w_pre"], out)
    x = c["x"].clone()
    x[1], x[2, 7], x[3, 9] = 0, math.nan, math.inf
    got = torch.empty_like(out)
    moe.moe_norm_forward(s, x, c["w_pre"], got)
    assert (got[1] == 0).all() and got[2].isnan().all()
    assert torch.equal(got[[0, 4, 5]], out[[0, 4, 5]])
    assert got[3, 9].isnan() and (got[3, :9] == 0).all()
    dx, dw = torch.empty_like(x), torch.empty(H, device=DEV)
    moe.moe_norm_backward(s, c["dnormed"], c["x"], c["w_pre"], dx, dw, ws)
    d2 = torch.empty_like(dx)
    moe.moe_norm_backward(s, c["dnormed"], x, c["w_pre"], d2, None, None)
    assert torch.equal(d2[[0, 4, 5]], dx[[0, 4, 5]]) and d2[2].isnan().all()
    zero = moe.NormShape(T=T, H=H, eps=0.0)
    moe.moe_norm_forward(zero, x, c["w_pre"], got)
    assert got[1].isnan().all()                              # 0 / 0, as the formula has it


def test_no_rows():
    s = moe.NormShape(T=0, H=64)
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    w = torch.ones(64, dtype=BF, device=DEV)
    a, b = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    moe.moe_norm_forward(s, e, w, e)
    moe.moe_norm_backward(s, e, e, w, e, a, None, y=e, w_post=w, dw_post=b)
    assert (a == 0).all() and (b == 0).all()


def test_many_rows_and_a_graph():
    """More rows than workgroups keep sums for, in a replayed graph with eager work between."""
    T, H = 3001, 1024
    c = _case(T, H, F32, 15)
    s = moe.NormShape(T=T, H=H, eps=1e-5, block_scale=0.3)
    ws = moe.alloc_norm_workspace(s, DEV)
    kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
    res, normed = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    o = dict(dx=torch.empty_like(res), dw_pre=torch.empty(H, device=DEV), dy=torch.empty_like(res),
             dw_post=torch.empty(H, device=DEV), dgate=torch.empty(T, device=DEV))

    def step():
        moe.moe_norm_forward(s, c["x"], c["w_pre"], normed, res=res, **kw)
        moe.moe_norm_backward(s, c["dnormed"], res, c["w_pre"], o["dx"], o["dw_pre"], ws,
                              dres=c["dres"], dy=o["dy"], dw_post=o["dw_post"], dgate=o["dgate"],
                              **kw)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    r = ffn_ref.norm_backward(c["dnormed"], c["dres"], res, c["w_pre"], 1e-5, 1.0, 0.3, **kw)
    first = None
    for k in range(3):
        for t in o.values():
            t.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, (v, b) in r.items():
            assert_close(o[n], v, b, "%s %d" % (n, k))
        now = {n: t.clone() for n, t in o.items()}
        assert first is None or all(torch.equal(first[n], now[n]) for n in now)
        first = now


def test_rows_past_32_bits():
    T, H = 300_000, 8192                                     # 2.5e9 bf16 values
    g = _gen(16)
    s = moe.NormShape(T=T, H=H)
    x = torch.zeros(T, H, dtype=BF, device=DEV)
    rows = torch.tensor([0, 262_143, 262_144, T - 1], device=DEV)
    x[rows] = _rows(g, BF, len(rows), H)
    w = (1 + _rows(g, F32, 1, H, 0.2)[0]).to(BF)
    out = torch.full_like(x, 5.0)
    moe.moe_norm_forward(s, x, w, out)
    n, off = ffn_ref.norm_of(x[rows], w, 1e-6)
    assert_close(out[rows], n, off, "normed")
    dn = torch.zeros_like(x)
    dn[rows] = _rows(g, BF, len(rows), H)
    dw = torch.empty(H, device=DEV)
    moe.moe_norm_backward(s, dn, x, w, out, dw, moe.alloc_norm_workspace(s, DEV))
    r = ffn_ref.norm_backward(dn[rows], None, x[rows], w, 1e-6, 1.0, 1.0)
    assert_close(out[rows], *r["dx"], "dx")
    assert_close(dw, *r["dw_pre"], "dw_pre")
