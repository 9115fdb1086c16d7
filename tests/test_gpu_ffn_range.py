"""The feed-forward block and the joint at the ends of what their header allows."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe

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
