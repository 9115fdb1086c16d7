"""The rows' gradients written over the rows, and rows past 2^32 bytes, in buffers of
their own."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
from gpu_util import DEV, say
from test_gpu_rows import make, randn

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("T,H,K,E,local", [(3, 128, 8, 4, 2), (65, 1024, 6, 32, 8),
                                           (517, 7168, 7, 64, 64)])
def test_drows_in_place_of_rows(T, H, K, E, local, dt):
    """The same bits as into a buffer of its own; rows without a route keep theirs."""
    say("in place", T, H, K, dt)
    s, d, w, R, g = make(T, H, K, E, local, 0.1, seed=T)
    dout, rows = randn(g, (T, H), dt), randn(g, (R, H), dt)
    for wt in (w, None):
        there, apart = rows.clone(), rows.clone()
        dw, dw2 = torch.empty(T, K, device=DEV), torch.empty(T, K, device=DEV)
        moe.moe_unpermute_backward(s, dout, rows, wt, d.route_row, apart, dw)
        moe.moe_unpermute_backward(s, dout, there, wt, d.route_row, there, dw2)
        assert torch.equal(there, apart) and torch.equal(dw2, dw)


def test_gradients_past_32_bit_offsets():
    """Whole numbers, so that dw is exact; every slot's row of drows, and every dw."""
    T, H, K = 45000, 7168, 8
    s = moe.MoeShape(T=T, H=H, I=128, K=K, E_total=8, E_local=8)
    R = moe.moe_row_capacity(s)
    assert R * H * 2 > 1 << 32
    rr = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=DEV)   # the last rows first
    g = torch.Generator(device=DEV).manual_seed(1)
    small = lambda *shape: torch.empty(*shape, dtype=BF, device=DEV).random_(0, 3, generator=g).sub_(1)
    dout, rows = small(T, H), small(R, H)
    w = (2.0 ** -torch.arange(K, device=DEV).float()).expand(T, K).contiguous()
    drows, dw = torch.empty_like(rows), torch.empty_like(w)
    moe.moe_unpermute_backward(s, dout, rows, w, rr, drows, dw)
    for k in range(K):
        at = rr.reshape(T, K)[:, k].long()
        assert torch.equal(drows[at], dout * 2.0 ** -k)
        assert torch.equal(dw[:, k], (dout.float() * rows[at].float()).sum(1))
