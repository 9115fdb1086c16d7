"""The residual joint and its gradients at the ends of what its header allows: rows far from 1, eps 0
and next to it."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ffn_ref
import test_gpu_norm as base
from ops_ref import assert_close

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("size,eps", [(1e-14, 0.0), (1e-13, 0.0), (1e-13, 1e-30), (1e10, 1e-6),
                                      (1e14, 1e-6), (1e15, 0.0), (1e16, 1e-6)])
@pytest.mark.parametrize("T,H", [(5, 96), (3, 7168), (1100, 160)])
def test_rows_far_from_one(T, H, size, eps, dt):
    """rho(v) ^ 3 leaves float32's range long before rho and the gradients do."""
    c = base._case(T, H, dt, T + H)
    c["x"], c["y"] = c["x"] * size, c["y"] * size
    s = moe.NormShape(T=T, H=H, eps=eps, skip_scale=0.75, block_scale=0.4)
    o = dict(dx=torch.empty_like(c["x"]), dw_pre=torch.empty(H, device=DEV),
             dy=torch.empty_like(c["x"]), dw_post=torch.empty(H, device=DEV),
             dgate=torch.empty(T, device=DEV))
    kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
    # (without dres, beside which the gradient of large rows is nothing)
    moe.moe_norm_backward(s, c["dnormed"], c["x"], c["w_pre"], o["dx"], o["dw_pre"],
                          moe.alloc_norm_workspace(s, DEV), dy=o["dy"], dw_post=o["dw_post"],
                          dgate=o["dgate"], **kw)
    r = ffn_ref.norm_backward(c["dnormed"], None, c["x"], c["w_pre"], eps, 0.75, 0.4, **kw)
    for k, (v, b) in r.items():
        # dy of large rows goes by dr, which is as small as they are large, over their size
        # again: below the normal numbers of bf16 and float32 each is off by steps of 2^-133
        # and 2^-149, and a flushed one by 2^-126
        assert_close(o[k], v, b + (2.0 ** -125 if k == "dy" else 0.0), k)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("size,eps", [(1e-14, 0.0), (1e-13, 1e-30), (1e10, 1e-6), (1e16, 1e-6)])
@pytest.mark.parametrize("T,H", [(5, 96), (3, 7168)])
def test_the_joint_of_rows_far_from_one(T, H, size, eps, dt):
    c = base._case(T, H, dt, T * H)
    c["x"], c["y"] = c["x"] * size, c["y"] * size
    s = moe.NormShape(T=T, H=H, eps=eps, skip_scale=0.75, block_scale=0.4 * size)
    res, normed = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
    moe.moe_norm_forward(s, c["x"], c["w_pre"], normed, res=res, **kw)
    assert_close(res, *ffn_ref.norm_forward(c["x"], None, eps, 0.75, s.c().block_scale, **kw),
                 "res")
    assert_close(normed, *ffn_ref.norm_of(res, c["w_pre"], eps), "normed")


@pytest.mark.parametrize("dt", [BF, F32])
def test_zero_rows_with_a_small_eps(dt):
    """rho of a row of zeros is 1 / sqrt(eps): its gradients are rho times what comes in."""
    T, H, eps = 4, 512, 1e-28
    c = base._case(T, H, dt, 31)
    c["x"][1], c["y"][2] = 0, 0
    s = moe.NormShape(T=T, H=H, eps=eps, block_scale=0.5)
    dx, dy = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
    moe.moe_norm_backward(s, c["dnormed"], c["x"], c["w_pre"], dx, None, None, dres=c["dres"],
                          dy=dy, **kw)
    r = ffn_ref.norm_backward(c["dnormed"], c["dres"], c["x"], c["w_pre"], eps, 1.0, 0.5, **kw)
    assert_close(dx, *r["dx"], "dx")
    assert_close(dy, *r["dy"], "dy")


def test_gradients_of_open_and_shut_gates():
    """sigmoid'(gate) = s(gate) s(-gate): both factors keep their bits however far the gate is
    open; 1 - s(gate) has none of them left from 17 on."""
    T, H = 12, 512
    c = base._case(T, H, F32, 17)
    c["gate"] = torch.tensor([-80.0, -30, -20, -17, -10, 0, 10, 15, 17, 20, 30, 80], device=DEV)
    s = moe.NormShape(T=T, H=H, block_scale=0.5)
    dg = torch.empty(T, device=DEV)
    kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
    moe.moe_norm_backward(s, None, None, None, None, None, None, dres=c["dres"], dgate=dg, **kw)
    g, y, dr = c["gate"].double(), c["y"].double(), c["dres"].double()
    z = y * ffn_ref.rms(y, 1e-6) * c["w_post"].double()
    k = 0.5 / ((1 + torch.exp(g)) * (1 + torch.exp(-g)))
    # exp within 2 steps of 2^-23, the sum, the quotient: 6 of 2^-24 a factor, three products;
    # the sums as in every row's dot product
    m = (dr * z).abs().sum(1)
    assert_close(dg, k * (dr * z).sum(1), k * 2.0 ** -24 * (20 + 2 * (H + 40)) * m, "dgate")


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("T,H", [(6, 512), (7, 7168), (6, 96)])
def test_mx_rows_keep_what_is_not_finite(T, H, dt):
    """An infinity or NaN of normed is a NaN code and has no part in its block's exponent."""
    c = base._case(T, H, dt, T + H)
    s = moe.NormShape(T=T, H=H)
    c["x"][1, 5], c["x"][2, 40] = float("nan"), float("inf")
    w = c["w_pre"]
    w[33], w[64] = float("inf"), float("nan")     # whole columns of every row
    normed = torch.empty_like(c["x"])
    codes = torch.empty(T, H, dtype=torch.uint8, device=DEV)
    exps = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV)
    moe.moe_norm_forward(s, c["x"], w, normed, normed_fp8=codes, normed_scale=exps)
    there = normed.isfinite()
    assert not there[1].any() and not there[:, [33, 64]].any() and there[0].sum() == H - 2
    want, we = ffn_ref.mx_rows(torch.where(there, normed, 0.0))
    got, lost = codes.cpu(), ~there.cpu()
    assert ((got[lost] & 0x7f) == 0x7f).all()
    assert torch.equal(exps.cpu(), we)
    zero = (want & 0x7f) == 0
    want = torch.where(zero, 0, want)
    assert torch.equal(torch.where(zero, got & 0x7f, got)[~lost], want[~lost])
    alone, ae = torch.empty_like(codes), torch.empty_like(exps)
    moe.moe_norm_forward(s, c["x"], w, None, normed_fp8=alone, normed_scale=ae)
    assert torch.equal(alone, codes) and torch.equal(ae, exps)
