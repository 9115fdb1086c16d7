"""The logits' gradient written over the logits."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
from gpu_util import DEV, say
from test_gpu_route import BF, F32, HF, draw, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (33, 63, 2), (130, 384, 6), (11, 1024, 8)])
def test_dlogits_in_place_of_logits(T, E, K, dt, renorm):
    """The same bits as in a buffer of its own."""
    say("route in place", T, E, K, dt, renorm)
    logits = draw(T, E, dt, seed=T)
    s, ids, w = run(logits, K, renorm)
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(5)).to(DEV)
    apart, there = torch.empty_like(logits), logits.clone()
    moe.moe_route_backward(s, logits, ids, w, g, apart, renormalize=renorm)
    moe.moe_route_backward(s, there, ids, w, g, there, renormalize=renorm)
    assert torch.equal(there, apart)
