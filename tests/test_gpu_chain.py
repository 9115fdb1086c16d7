"""The router, the dispatch, the rows to their experts and back and the adapters one after
the other, as a training step and a serving step call them, against the same steps in
64 bits (and autograd's gradients of them)."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ops_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,H,E,local,begin,K,renorm", [(37, 256, 16, 16, 0, 3, True),
                                                        (260, 640, 64, 24, 8, 6, False),
                                                        (1, 128, 8, 8, 0, 2, True)])
def test_training_step(T, H, E, local, begin, K, renorm):
    """logits -> route -> dispatch -> permute -> an expert that scales its rows ->
    unpermute, and back to the gradients of the tokens and of the logits."""
    say("chain", T, H, E, local, begin, K, renorm)
    g = torch.Generator().manual_seed(T)
    x, dout = (torch.randn(T, H, generator=g).to(DEV) for _ in range(2))
    logits = torch.randn(T, E, generator=g).to(DEV)
    gain = 2.0 ** torch.randint(-2, 3, (local,), generator=g).float().to(DEV)
    s = moe.MoeShape(T=T, H=H, I=128, K=K, E_total=E, E_local=local, expert_begin=begin)
    R = moe.moe_row_capacity(s)
    ids = torch.empty(T, K, dtype=torch.int32, device=DEV)
    w = torch.empty(T, K, device=DEV)
    moe.moe_route(s, logits, ids, w, renormalize=renorm)
    d = moe.alloc_dispatch(s, DEV)
    moe.moe_dispatch(s, ids, d)
    rows = torch.zeros(R, H, device=DEV)
    moe.moe_permute(s, x, d.route_row, rows)
    # the expert of each row, from the dispatch's own tables
    used = int(d.offsets[local])
    expert = torch.repeat_interleave(torch.arange(local, device=DEV), d.counts.long())
    y = rows.clone()
    y[:used] *= gain[expert][:, None]
    out = torch.empty(T, H, device=DEV)
    moe.moe_unpermute(s, y, w, d.route_row, out)
    dy, dw = torch.zeros(R, H, device=DEV), torch.empty(T, K, device=DEV)
    moe.moe_unpermute_backward(s, dout, y, w, d.route_row, dy, dw)
    drows = dy.clone()
    drows[:used] *= gain[expert][:, None]
    dx, dlogits = torch.empty_like(x), torch.empty_like(logits)
    moe.moe_permute_backward(s, drows, d.route_row, dx)
    moe.moe_route_backward(s, logits, ids, w, dw, dlogits, renormalize=renorm)

    x64 = x.cpu().double().requires_grad_()
    l64 = logits.cpu().double().requires_grad_()
    i64 = ids.cpu().long()
    p = torch.softmax(l64, 1)
    # renormalised: the softmax of the chosen logits themselves, so that the others'
    # gradient is 0 and not what two 64-bit terms leave of each other
    w64 = torch.softmax(torch.gather(l64, 1, i64), 1) if renorm else torch.gather(p, 1, i64)
    here = (i64 >= begin) & (i64 < begin + local)
    of = torch.where(here, gain.cpu().double()[(i64 - begin).clamp(0, local - 1)], 0.0)
    per = (w64 * of).sum(1)
    want = per[:, None] * x64
    (want * dout.cpu().double()).sum().backward()
    # each of the chain's few float32 steps rounds once; sums of K rows, of H
    # products (dw) and of a softmax over E: all within (H + E + 60) 2^-24 of
    # their terms' magnitudes
    u = ref.U32 * (H + E + 60)
    mag = (w64.detach().abs() * of.abs()).sum(1)[:, None]
    ref.assert_close(out, want.detach(), u * mag * x64.detach().abs(), "out")
    ref.assert_close(dx, x64.grad, u * mag * dout.cpu().double().abs(), "dx")
    dots = (x64.detach().abs() * dout.cpu().double().abs()).sum(1, keepdim=True) * 4
    scale = p.detach() if not renorm else torch.zeros_like(p).scatter(1, i64, w64.detach())
    ref.assert_close(dlogits, l64.grad, 4 * u * scale * dots, "dlogits")


def test_serving_step():
    """Router logits through the shared projection with adapters, the rows of each expert
    through an adapter of their own beside a given base, and back."""
    T, H, E, K, L, r = 70, 256, 32, 4, 5, 16
    g = torch.Generator().manual_seed(3)
    rn = lambda *shape, std=1.0: (torch.randn(*shape, generator=g) * std).to(BF).to(DEV)
    x, wr = rn(T, H), rn(E, H, std=H ** -0.5)
    a, b = rn(L, r, H, std=H ** -0.5), rn(L, E, r, std=r ** -0.5)
    ids_a = torch.randint(-1, L, (T,), generator=g).to(torch.int32).to(DEV)
    pa = moe.AdapterShape(T=T, H=H, N=E, L=L, rank=r)
    logits = torch.empty(T, E, dtype=BF, device=DEV)
    moe.moe_adapter_project(pa, x, wr, ids_a, a, b, None, logits,
                            moe.alloc_adapter_workspace(pa, DEV))
    want, off = ref.adapters(x, wr, None, ids_a, a, b, None)
    ref.assert_close(logits, want, off, "logits")
    s = moe.MoeShape(T=T, H=H, I=128, K=K, E_total=E, E_local=E)
    ids = torch.empty(T, K, dtype=torch.int32, device=DEV)
    w = torch.empty(T, K, device=DEV)
    moe.moe_route(s, logits, ids, w)
    rid, rw, _, _ = ref.route(logits, K, True)
    assert torch.equal(ids.cpu(), torch.from_numpy(rid))
    d = moe.alloc_dispatch(s, DEV)
    moe.moe_dispatch(s, ids, d)
    R = moe.moe_row_capacity(s)
    rows = torch.zeros(R, H, dtype=BF, device=DEV)
    moe.moe_permute(s, x, d.route_row, rows)
    # an adapter per expert on its rows, added to the rows themselves
    ea, eb = rn(E, r, H, std=H ** -0.5), rn(E, H, r, std=r ** -0.5)
    expert = torch.repeat_interleave(torch.arange(E, device=DEV), d.counts.long())
    pe = moe.AdapterShape(T=R, H=H, N=H, L=E, rank=r)
    y = torch.empty_like(rows)
    moe.moe_adapter_project(pe, rows, None, expert.to(torch.int32), ea, eb, None, y,
                            moe.alloc_adapter_workspace(pe, DEV), base=rows)
    want, off = ref.adapters(rows, None, rows, expert, ea, eb, None)
    ref.assert_close(y, want, off, "rows")
    out = torch.empty_like(x)
    moe.moe_unpermute(s, y, w, d.route_row, out)
    o, mag = ref.unpermute(y, w, d.route_row, T, K)
    ref.assert_close(out, o, (K + 1) * ref.U32 * mag, "out")
