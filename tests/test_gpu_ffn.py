"""The dense feed-forward block on the GPU: whole numbers to the bit at sizes for every kernel
and edge, normal ones inside derived bounds, both forms of what is kept, and the gradients."""

import math

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ffn_ref
from ops_ref import assert_close

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16
DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).double()


def _normal(g, dt, std, *shape):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)


def _round(v, dt):
    """float64 whole numbers (or halves) to dt: exact in float32 first."""
    assert (v.float().double() == v).all()
    return v.float().to(dt)


# T, H, I: single tokens, the edges of 16, 32, 64 and 128 rows and columns, odd tails, K that
# is one step, a ragged one, or split in parts; wide enough for tiles of 256 (8,192 x 2,048
# columns of gate and up: 256 tiles and more, and what is left over in halves)
SIZES = [(1, 32, 32), (1, 2048, 512), (2, 96, 160), (7, 160, 96), (15, 512, 64), (16, 64, 512),
         (17, 544, 288), (31, 1056, 32), (33, 32, 1056), (63, 256, 256), (64, 2304, 96),
         (65, 128, 672), (100, 1024, 512), (127, 96, 96), (128, 1024, 2048), (129, 288, 160),
         (191, 736, 544), (256, 512, 512), (257, 1632, 352), (513, 128, 1408),
         (1000, 2304, 160), (2100, 96, 4192), (4129, 2080, 2112), (8200, 64, 1120)]


def _whole(T, H, I, dt, seed):
    """x, w13, w2 whole numbers with every gate at or above the limit of 16 (silu(16) is 16 to
    2^-23 of it), every sum exact in float32 and h exact in dt."""
    g = _gen(seed)
    x = _ints(g, 0, 1, T, H)
    x[:, 0] = 16
    wg = _ints(g, 0, 2, I, H)
    wg[:, 0] = 1
    wu = torch.where(torch.rand(I, H, generator=g, device=DEV) < 8 / H, _ints(g, -1, 1, I, H), 0.0)
    wu[:, 0] = 0
    w2 = torch.where(torch.rand(H, I, generator=g, device=DEV) < 0.5, _ints(g, -1, 1, H, I), 0.0)
    return x.to(dt), torch.cat([wg, wu]).to(dt), w2.to(dt)


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_forward_whole_numbers(T, H, I, dt):
    x, w13, w2 = _whole(T, H, I, dt, T + H + I)
    s = moe.FfnShape(T=T, H=H, I=I, gate_limit=16.0, up_limit=7.0)
    ws = moe.alloc_ffn_workspace(s, DEV)
    gu = x.double() @ w13.double().t()
    h = 16.0 * gu[:, I:].clamp(-7, 7)
    want = h @ w2.double().t()
    out = torch.full((T + 1, H), -3.0, dtype=dt, device=DEV)
    kept = torch.full((T + 1, 2 * I), -3.0, dtype=dt, device=DEV)
    moe.moe_ffn_forward(s, x, w13, w2, out[:T], ws, gate_up=kept[:T])
    assert torch.equal(out[:T], _round(want, dt))
    assert torch.equal(kept[:T], _round(gu, dt))
    assert (out[T] == -3).all() and (kept[T] == -3).all()
    # added to what the experts gave, in place
    base = _ints(_gen(1), -50, 50, T, H).to(dt)
    moe.moe_ffn_forward(s, x, w13, w2, base2 := base.clone(), ws, base=base2)
    assert torch.equal(base2, _round(want + base.double(), dt))
    # 8 bits kept: the codes and exponents of the exact sums
    codes = torch.full((T + 1, 2 * I), 77, dtype=torch.uint8, device=DEV)
    exps = torch.full((T + 1, 2 * I // 32), 77, dtype=torch.uint8, device=DEV)
    moe.moe_ffn_forward(s, x, w13, w2, out[:T], ws, gate_up=codes[:T], gate_up_scale=exps[:T])
    assert torch.equal(out[:T], _round(want, dt))
    c, e = ffn_ref.mx_rows(gu)
    assert torch.equal(exps[:T].cpu(), e)
    zero = (c & 0x7f) == 0                                # a 0 may come with either sign
    got = codes[:T].cpu()
    assert torch.equal(torch.where(zero, got & 0x7f, got), torch.where(zero, 0, c))
    assert (codes[T] == 77).all() and (exps[T] == 77).all()


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_backward_whole_numbers(T, H, I, dt):
    """Kept gates at 16 (silu 16, its slope 1 to 2^-18) or above the limit (slope 0)."""
    g = _gen(T + H + I + 1)
    x, w13 = _ints(g, -2, 2, T, H), _ints(g, -1, 1, 2 * I, H)
    w2 = torch.where(torch.rand(H, I, generator=g, device=DEV) < 4 / H, _ints(g, -1, 1, H, I), 0.0)
    dout = _ints(g, -1, 1, T, H)
    gate = torch.where(torch.rand(T, I, generator=g, device=DEV) < 0.7, 16.0, 24.0)
    up = _ints(g, -5, 5, T, I)
    dh = dout @ w2
    uc = up.clamp(-4, 4)
    dg = torch.where(gate > 16, 0.0, dh * uc)
    du = torch.where(up.abs() > 4, 0.0, 16 * dh)
    q = torch.cat([dg, du], 1)
    assert (q.to(dt).double() == q).all()
    want = [q @ w13, q.t() @ x, dout.t() @ (16 * uc)]
    s = moe.FfnShape(T=T, H=H, I=I, gate_limit=16.0, up_limit=4.0)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    kept = torch.cat([gate, up], 1)
    args = [t.to(dt).contiguous() for t in (dout, x, w13, w2, kept)]

    def outs(wdt=dt):
        return [torch.full((T + 1, H), -3.0, dtype=dt, device=DEV),
                torch.full((2 * I + 1, H), -3.0, dtype=wdt, device=DEV),
                torch.full((H + 1, I), -3.0, dtype=wdt, device=DEV)]

    o = outs()
    moe.moe_ffn_backward(s, *args, *[t[:-1] for t in o], ws)
    for t, w in zip(o, want):
        assert torch.equal(t[:-1], _round(w, dt)) and (t[-1] == -3).all()
    # float32 gradients, added to what is there; x and the pre-activations in 8 bits
    o = outs(torch.float32)
    c, e = ffn_ref.mx_rows(kept)
    cx, ex = ffn_ref.mx_rows(x)
    if float((ffn_ref.mx_values(c, e) - kept.cpu()).abs().max()) > 0:
        pytest.fail("the kept values are not exact in 8 bits")
    moe.moe_ffn_backward(s, args[0], cx.to(DEV), *args[2:4], c.to(DEV), *[t[:-1] for t in o], ws,
                         gate_up_scale=e.to(DEV), x_scale=ex.to(DEV), accumulate=True)
    assert torch.equal(o[0][:-1], _round(want[0], dt))
    for t, w in zip(o[1:], want[1:]):
        assert torch.equal(t[:-1].double(), w - 3) and (t[-1] == -3).all()


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("T,H,I,lim", [(1, 512, 256, 10.0), (5, 1056, 96, 1.0), (33, 288, 544, 2.0),
                                       (130, 1024, 512, math.inf), (700, 512, 1408, 3.0),
                                       (2500, 256, 3584, 10.0)])
def test_normal_values(T, H, I, lim, dt):
    g = _gen(T + I)
    x, w13 = _normal(g, dt, 1, T, H), _normal(g, dt, 1.5 * H ** -0.5, 2 * I, H)
    w2, dout = _normal(g, dt, I ** -0.5, H, I), _normal(g, dt, 1, T, H)
    base = _normal(g, dt, 1, T, H)
    s = moe.FfnShape(T=T, H=H, I=I, gate_limit=lim, up_limit=lim)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    out, kept = torch.empty_like(x), torch.empty(T, 2 * I, dtype=dt, device=DEV)
    moe.moe_ffn_forward(s, x, w13, w2, out, ws, base=base, gate_up=kept)
    ref, off, gu, gu_off = ffn_ref.ffn_forward(x, w13, w2, lim, lim, base)
    assert_close(out, ref, off, "out")
    assert_close(kept, gu, gu_off, "gate_up")
    codes = torch.empty(T, 2 * I, dtype=torch.uint8, device=DEV)
    exps = torch.empty(T, 2 * I // 32, dtype=torch.uint8, device=DEV)
    out2 = torch.empty_like(out)
    moe.moe_ffn_forward(s, x, w13, w2, out2, ws, base=base, gate_up=codes, gate_up_scale=exps)
    assert torch.equal(out, out2)
    cx, ex = [t.to(DEV) for t in ffn_ref.mx_rows(x)]
    for eight in (False, True):
        dx, dw13, dw2 = torch.empty_like(x), torch.empty_like(w13), torch.empty_like(w2)
        if eight:
            xv, guv = ffn_ref.mx_values(cx, ex).to(DEV), ffn_ref.mx_values(codes, exps).to(DEV)
            moe.moe_ffn_backward(s, dout, cx, w13, w2, codes, dx, dw13, dw2, ws,
                                 gate_up_scale=exps, x_scale=ex)
        else:
            xv, guv = x, kept
            moe.moe_ffn_backward(s, dout, x, w13, w2, kept, dx, dw13, dw2, ws)
        r = ffn_ref.ffn_backward(dout, xv, w13, w2, guv, lim, lim, dt)
        assert_close(dx, r[0], r[1], "dx %s" % eight)
        assert_close(dw13, r[2], r[3], "dw13 %s" % eight)
        assert_close(dw2, r[4], r[5], "dw2 %s" % eight)


def test_some_gradients_only():
    """Each gradient alone is the one of the full call, bit for bit; the rest is untouched."""
    T, H, I = 77, 160, 96
    g = _gen(9)
    x, w13, w2 = _normal(g, BF, 1, T, H), _normal(g, BF, 0.1, 2 * I, H), _normal(g, BF, 0.1, H, I)
    dout, kept = _normal(g, BF, 1, T, H), _normal(g, BF, 1, T, 2 * I)
    s = moe.FfnShape(T=T, H=H, I=I)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    full = [torch.empty_like(t) for t in (x, w13, w2)]
    moe.moe_ffn_backward(s, dout, x, w13, w2, kept, *full, ws)
    for i in range(3):
        ws.fill_(255)
        o = [torch.empty_like(t) if k == i else None for k, t in enumerate(full)]
        moe.moe_ffn_backward(s, dout, x if i == 1 else None, w13 if i == 0 else None, w2, kept,
                             *o, ws)
        assert torch.equal(o[i], full[i])
    # 16-bit gradients added to what is there
    acc = [None, full[1].clone(), full[2].clone()]
    moe.moe_ffn_backward(s, dout, x, w13, w2, kept, *acc, ws, accumulate=True)
    for i in (1, 2):
        r = ffn_ref.ffn_backward(dout, x, w13, w2, kept, 10.0, 10.0, BF)
        assert_close(acc[i], r[2 * i] + full[i].double(),
                     r[2 * i + 1] + 2 ** -23 * full[i].double().abs(), "accumulate %d" % i)


def test_no_rows():
    s = moe.FfnShape(T=0, H=64, I=32)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    x, w13 = torch.empty(0, 64, dtype=BF, device=DEV), torch.ones(64, 64, dtype=BF, device=DEV)
    w2, kept = torch.ones(64, 32, dtype=BF, device=DEV), torch.empty(0, 64, dtype=BF, device=DEV)
    moe.moe_ffn_forward(s, x, w13, w2, x, ws)
    for wdt in (BF, torch.float32):
        for acc in (False, True):
            a, b = torch.ones(64, 64, dtype=wdt, device=DEV), torch.ones(64, 32, dtype=wdt, device=DEV)
            moe.moe_ffn_backward(s, x, x, w13, w2, kept, x, a, b, ws, accumulate=acc)
            assert (a == (1 if acc else 0)).all() and (b == (1 if acc else 0)).all()


@pytest.mark.parametrize("T", [3, 40, 200])
def test_infinities_and_nan_stay_in_their_rows(T):
    """A row of NaN, one of +inf products and one of -inf gates: the other rows' bits do not
    change, a NaN comes out as one, a gate of +inf is the limit's."""
    H, I = 288, 160
    g = _gen(11)
    x, w13, w2 = _normal(g, BF, 1, T, H), _normal(g, BF, 0.1, 2 * I, H), _normal(g, BF, 0.1, H, I)
    s = moe.FfnShape(T=T, H=H, I=I)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    out, kept = torch.empty_like(x), torch.empty(T, 2 * I, dtype=BF, device=DEV)
    moe.moe_ffn_forward(s, x, w13, w2, out, ws, gate_up=kept)
    x2 = x.clone()
    x2[1, 5] = math.nan
    out2, kept2 = torch.empty_like(out), torch.empty_like(kept)
    moe.moe_ffn_forward(s, x2, w13, w2, out2, ws, gate_up=kept2)
    rest = [t for t in range(T) if t != 1]
    assert out2[1].isnan().all() and kept2[1].isnan().all()
    assert torch.equal(out2[rest], out[rest]) and torch.equal(kept2[rest], kept[rest])
    # gradients: an infinite kept gate is above its limit: no gradient of its own, and the
    # limit's silu for u; a NaN in dout reaches its row of dx and every weight, no other row
    kept3 = kept.clone()
    kept3[2, :I] = math.inf
    dout = _normal(g, BF, 1, T, H)
    got = [torch.empty_like(t) for t in (x, w13, w2)]
    moe.moe_ffn_backward(s, dout, x, w13, w2, kept3, *got, ws)
    finite = kept3.clone()
    finite[2, :I] = 11.0
    r = ffn_ref.ffn_backward(dout, x, w13, w2, finite, 10.0, 10.0, BF)
    for i in range(3):
        assert_close(got[i], r[2 * i], r[2 * i + 1], "inf gate %d" % i)
    dx = torch.empty_like(x)
    dout[0, 3] = math.nan
    moe.moe_ffn_backward(s, dout, None, w13, w2, kept3, dx, None, None, ws)
    assert dx[0].isnan().all() and torch.equal(dx[1:], got[0][1:])


def test_graph_streams_and_repeats():
    """Captured on a side stream, replayed several times with eager work between: the eager
    call's bits, forward and backward, both forms of what is kept."""
    T, H, I = 130, 544, 288
    g = _gen(12)
    x, w13, w2 = _normal(g, BF, 1, T, H), _normal(g, BF, 0.1, 2 * I, H), _normal(g, BF, 0.1, H, I)
    dout = _normal(g, BF, 1, T, H)
    s = moe.FfnShape(T=T, H=H, I=I)

    def buffers():
        return dict(out=torch.zeros_like(x), kept=torch.zeros(T, 2 * I, dtype=torch.uint8, device=DEV),
                    exps=torch.zeros(T, 2 * I // 32, dtype=torch.uint8, device=DEV),
                    dx=torch.zeros_like(x), dw13=torch.zeros(2 * I, H, device=DEV),
                    dw2=torch.zeros(H, I, device=DEV),
                    ws=moe.alloc_ffn_workspace(s, DEV, backward=True))

    def step(b):
        moe.moe_ffn_forward(s, x, w13, w2, b["out"], b["ws"], gate_up=b["kept"],
                            gate_up_scale=b["exps"])
        moe.moe_ffn_backward(s, dout, x, w13, w2, b["kept"], b["dx"], b["dw13"], b["dw2"], b["ws"],
                             gate_up_scale=b["exps"])

    eager, b = buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(b)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step(b)
    for k in range(4):
        for n in ("out", "dx", "dw13", "dw2"):
            b[n].fill_(7)
        x.mul_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("out", "kept", "exps", "dx", "dw13", "dw2"):
            assert torch.equal(b[n], eager[n]), (k, n)


def test_two_calls_at_once():
    """Two streams, a workspace each: the bits of the calls one after the other."""
    g = _gen(13)
    T, H, I = 600, 1024, 512
    s = moe.FfnShape(T=T, H=H, I=I)
    sets = []
    for k in range(2):
        sets.append(dict(x=_normal(g, BF, 1, T, H), w13=_normal(g, BF, 0.1, 2 * I, H),
                         w2=_normal(g, BF, 0.1, H, I), out=torch.empty(T, H, dtype=BF, device=DEV),
                         ws=moe.alloc_ffn_workspace(s, DEV)))
    want = []
    for b in sets:
        moe.moe_ffn_forward(s, b["x"], b["w13"], b["w2"], b["out"], b["ws"])
        want.append(b["out"].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for b, st in zip(sets, streams):
            b["out"].zero_()
        torch.cuda.synchronize()
        for b, st in zip(sets, streams):
            moe.moe_ffn_forward(s, b["x"], b["w13"], b["w2"], b["out"], b["ws"], stream=st)
        torch.cuda.synchronize()
        for b, w in zip(sets, want):
            assert torch.equal(b["out"], w)


def test_rows_past_32_bits():
    """x, out and their gradients of more than 2^32 bytes and 2^31 values: the last rows are
    right, and so are the weights' gradients, to which only a few rows contribute."""
    T, H, I = 140_001, 16_384, 32
    g = _gen(14)
    s = moe.FfnShape(T=T, H=H, I=I)
    x = torch.zeros(T, H, dtype=BF, device=DEV)
    rows = torch.tensor([0, 65_535, 131_071, 131_072, T - 2, T - 1], device=DEV)
    x[rows] = _normal(g, BF, 1, len(rows), H)
    dout = torch.zeros(T, H, dtype=BF, device=DEV)
    dout[rows] = _normal(g, BF, 1, len(rows), H)
    w13, w2 = _normal(g, BF, 0.01, 2 * I, H), _normal(g, BF, 0.2, H, I)
    out, dx = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    kept = torch.empty(T, 2 * I, dtype=BF, device=DEV)
    dw13, dw2 = torch.empty_like(w13), torch.empty_like(w2)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    moe.moe_ffn_forward(s, x, w13, w2, out, ws, gate_up=kept)
    moe.moe_ffn_backward(s, dout, x, w13, w2, kept, dx, dw13, dw2, ws)
    ref, off, gu, gu_off = ffn_ref.ffn_forward(x[rows], w13, w2, 10.0, 10.0)
    assert_close(out[rows], ref, off, "out")
    r = ffn_ref.ffn_backward(dout[rows], x[rows], w13, w2, kept[rows], 10.0, 10.0, BF)
    assert_close(dx[rows], r[0], r[1], "dx")
    assert_close(dw13, r[2], r[3], "dw13")
    assert_close(dw2, r[4], r[5], "dw2")
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[rows] = False
    for t in (out, dx):
        assert not bool((t.abs().amax(1) * rest).any())
