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
