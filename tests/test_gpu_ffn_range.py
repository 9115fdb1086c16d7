"""The feed-forward block and the joint at the ends of what their header allows."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ffn_ref
import test_gpu_ffn as base
from ops_ref import HALF, U32, assert_close

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16
DEV = "cuda"


def test_no_rows_and_frozen_weights():
    """An expert's or a rank's empty batch: dx alone, and each of the joint's row gradients."""
    e, w = torch.empty(0, 64, dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV)
    s = moe.FfnShape(T=0, H=64, I=32)
    w13, w2 = torch.ones(64, 64, dtype=BF, device=DEV), torch.ones(64, 32, dtype=BF, device=DEV)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    moe.moe_ffn_backward(s, e, None, w13, w2, e, e, None, None, ws)
    n = moe.NormShape(T=0, H=64)
    none = torch.empty(0, device=DEV)
    moe.moe_norm_backward(n, e, e, w, e, None, None)
    moe.moe_norm_backward(n, None, None, None, None, None, None, dres=e, y=e, w_post=w, gate=none,
                          dy=e, dgate=none)


def test_a_workspace_serves_fewer_rows():
    """One workspace for the largest batch, calls of fewer rows that go in parts of K: the bits
    that a workspace of their own gives."""
    H, I, most = 2304, 1408, 1200
    g = torch.Generator(device=DEV)
    g.manual_seed(41)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dout = n(most, H).to(BF), n(most, H).to(BF)
    w13, w2 = (n(2 * I, H) * H ** -0.5).to(BF), (n(H, I) * I ** -0.5).to(BF)
    large = moe.alloc_ffn_workspace(moe.FfnShape(T=most, H=H, I=I), DEV, backward=True)
    only = moe.alloc_ffn_workspace(moe.FfnShape(T=most, H=H, I=I), DEV)
    for T in (most, 256, 192, 128, 65, 64, 20):
        s = moe.FfnShape(T=T, H=H, I=I)
        own = moe.alloc_ffn_workspace(s, DEV, backward=True)
        results = []
        for ws in (own, large, only):
            out, kept = torch.empty(T, H, dtype=BF, device=DEV), torch.empty(T, 2 * I, dtype=BF,
                                                                             device=DEV)
            moe.moe_ffn_forward(s, x[:T], w13, w2, out, ws, gate_up=kept)
            grads = [torch.empty_like(t) for t in (out, w13, w2)]
            if ws is not only:
                moe.moe_ffn_backward(s, dout[:T], x[:T], w13, w2, kept, *grads, ws)
            results.append([out, kept] + (grads if ws is not only else []))
        for r in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], r)), T


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("dt", [BF, F16])
def test_an_exponent_byte_of_255_is_nan(T, dt):
    """E8M0 255 stands for NaN, as in the experts' products: the whole block of 32 values, in
    x as the experts take it and in what was kept."""
    H, I, row = 96, 64, T // 2
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dt)  # noqa: E731
    dout, w13, w2 = n(T, H), n(2 * I, H), n(H, I)
    s = moe.FfnShape(T=T, H=H, I=I)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    # codes of 0 and of 1 and -1 in turn, of exponent 0
    code = torch.tensor([0x00, 0x38, 0xb8], dtype=torch.uint8, device=DEV)
    x = code[torch.arange(T * H, device=DEV).reshape(T, H) % 3]
    kept = code[torch.arange(T * 2 * I, device=DEV).reshape(T, 2 * I) % 3]
    xs = torch.full((T, H // 32), 127, dtype=torch.uint8, device=DEV)
    ks = torch.full((T, 2 * I // 32), 127, dtype=torch.uint8, device=DEV)
    xs[row, 1], ks[3, 2] = 255, 255                     # columns 32 .. 63; u of 0 .. 31
    dx, dw13, dw2 = torch.empty_like(dout), torch.empty_like(w13), torch.empty_like(w2)
    moe.moe_ffn_backward(s, dout, x, w13, w2, kept, dx, dw13, dw2, ws, gate_up_scale=ks,
                         x_scale=xs)
    nan = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    nan[3] = True                                       # dg of a NaN u
    assert torch.equal(dx.isnan(), nan) and dx[~nan].isfinite().all()
    nan = torch.zeros(2 * I, H, dtype=torch.bool, device=DEV)
    nan[:, 32:64] = True
    nan[:32] = True                                     # its dg (du has no u in it)
    assert torch.equal(dw13.isnan(), nan) and dw13[~nan].isfinite().all()
    nan = torch.zeros(H, I, dtype=torch.bool, device=DEV)
    nan[:, :32] = True                                  # its h
    assert torch.equal(dw2.isnan(), nan) and dw2[~nan].isfinite().all()


@pytest.mark.parametrize("T", [4, 40, 200, 700])
@pytest.mark.parametrize("dt", [BF, F16])
def test_infinite_rows(T, dt):
    """Infinite x: a gate of +inf is the limit's, an up of -inf its own limit's, a gate of
    -inf NaN (-inf / inf, as the formula has it); no other row's bits change."""
    H, I, lim = 288, 160, 10.0
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, w13, w2 = n(T, H).to(dt), (n(2 * I, H) * 0.1).to(dt), (n(H, I) * 0.1).to(dt)
    w13[:I, 0], w13[I:, 0] = 0.5, -0.5
    s = moe.FfnShape(T=T, H=H, I=I, gate_limit=lim, up_limit=lim)
    ws = moe.alloc_ffn_workspace(s, DEV)
    results = []
    for infinite in (False, True):
        v = x.clone()
        if infinite:
            v[1, 0], v[2, 0] = float("inf"), -float("inf")
        out, kept = torch.empty_like(x), torch.empty(T, 2 * I, dtype=dt, device=DEV)
        moe.moe_ffn_forward(s, v, w13, w2, out, ws, gate_up=kept)
        results.append((out, kept))
    (a, ak), (b, bk) = results
    rest = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(a[rest], b[rest]) and torch.equal(ak[rest], bk[rest])
    inf = float("inf")
    assert (bk[1, :I] == inf).all() and (bk[1, I:] == -inf).all()
    assert (bk[2, :I] == -inf).all() and (bk[2, I:] == inf).all() and b[2].isnan().all()
    # silu(10) within 12 + 10 steps of 2^-24, times -10, rounded once; the sum over I
    h = torch.full((I,), -lim * lim / (1 + 2.718281828459045 ** -lim), dtype=torch.float64,
                   device=DEV)
    h_off = h.abs() * (HALF[dt] * (1 + 2.0 ** -10) + 24 * U32)
    want = w2.double() @ h
    off = w2.double().abs() @ (h_off + (I + 2) * U32 * (h.abs() + h_off))
    assert_close(b[1], want, off, "the limits' row")


def test_graph_writes_what_is_kept():
    """What the forward pass keeps in 8 bits, cleared before every replay, and the gradients
    that read it: the eager call's bits."""
    T, H, I = 130, 544, 288
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dout = n(T, H).to(BF), n(T, H).to(BF)
    w13, w2 = (n(2 * I, H) * 0.1).to(BF), (n(H, I) * 0.1).to(BF)
    s = moe.FfnShape(T=T, H=H, I=I)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    o = dict(out=torch.empty_like(x), dx=torch.empty_like(x),
             kept=torch.empty(T, 2 * I, dtype=torch.uint8, device=DEV),
             exps=torch.empty(T, 2 * I // 32, dtype=torch.uint8, device=DEV),
             dw13=torch.empty(2 * I, H, device=DEV), dw2=torch.empty(H, I, device=DEV))

    def step():
        moe.moe_ffn_forward(s, x, w13, w2, o["out"], ws, gate_up=o["kept"],
                            gate_up_scale=o["exps"])
        moe.moe_ffn_backward(s, dout, x, w13, w2, o["kept"], o["dx"], o["dw13"], o["dw2"], ws,
                             gate_up_scale=o["exps"])

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        want = {k: t.clone() for k, t in o.items()}
        with torch.cuda.graph(graph, stream=side):
            step()
    for k in range(4):
        for t in (*o.values(), ws):
            t.fill_(99)
        x.mul_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, t in o.items():
            assert torch.equal(t, want[name]), (k, name)


@pytest.mark.parametrize("T", [96, 385])
def test_a_dense_layers_width(T):
    """I wider than H by more than twice, as a dense layer beside expert layers has it."""
    H, I, lim = 7168, 18432, 10.0
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dout = n(T, H).to(BF), n(T, H).to(BF)
    w13, w2 = (n(2 * I, H) * H ** -0.5).to(BF), (n(H, I) * I ** -0.5).to(BF)
    s = moe.FfnShape(T=T, H=H, I=I, gate_limit=lim, up_limit=lim)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    out, kept = torch.empty_like(x), torch.empty(T, 2 * I, dtype=BF, device=DEV)
    moe.moe_ffn_forward(s, x, w13, w2, out, ws, gate_up=kept)
    ref, off, gu, gu_off = ffn_ref.ffn_forward(x, w13, w2, lim, lim)
    assert_close(out, ref, off, "out")
    assert_close(kept, gu, gu_off, "gate_up")
    del ref, off, gu, gu_off
    dx, dw13, dw2 = torch.empty_like(x), torch.empty_like(w13), torch.empty_like(w2)
    moe.moe_ffn_backward(s, dout, x, w13, w2, kept, dx, dw13, dw2, ws)
    r = ffn_ref.ffn_backward(dout, x, w13, w2, kept, lim, lim, BF)
    assert_close(dx, r[0], r[1], "dx")
    some, cols = slice(None, None, 61), slice(None, None, 7)
    assert_close(dw13[some, cols], r[2][some, cols], r[3][some, cols], "dw13")
    assert_close(dw2[some, cols], r[4][some, cols], r[5][some, cols], "dw2")


def test_as_many_rows_as_the_layer_takes():
    """65,536 rows, the layer's own largest batch, forward and backward."""
    base.test_forward_whole_numbers(65536, 512, 256, BF)
    base.test_backward_whole_numbers(65536, 512, 256, F16)
