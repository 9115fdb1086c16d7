"""Rows to their experts and back, with gradients, against the 64-bit definition."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ops_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def make(T, H, K, E, local, pad, mode=0, cap=0, seed=0, begin=0):
    g = torch.Generator().manual_seed(seed)
    s = moe.MoeShape(T=T, H=H, I=128, K=K, E_total=E, E_local=local, expert_begin=begin,
                     dispatch_mode=mode, capacity=cap)
    ids = torch.randint(0, E, (T, K), generator=g)
    ids[torch.rand(T, K, generator=g) < pad] = -1
    if T > 2:
        ids[1] = -1                               # a token that goes nowhere
        ids[2] = ids[2, 0]                        # the same expert in every slot
    d = moe.alloc_dispatch(s, DEV)
    moe.moe_dispatch(s, ids.to(torch.int32).to(DEV), d)
    w = torch.rand(T, K, generator=g)
    w[(ids < begin) | (ids >= begin + local)] = float("nan")   # skipped slots' weights
    R = max(moe.moe_row_capacity(s), 1)
    return s, d, w.to(DEV), R, g


def randn(g, shape, dt):
    return torch.randn(shape, generator=g).to(dt).to(DEV)


CASES = [
    # T, H, K, E, local, pad, mode, cap, begin
    (1, 128, 1, 1, 1, 0.0, 0, 0, 0),
    (1, 7168, 6, 384, 48, 0.0, 0, 0, 0),
    (3, 128, 8, 4, 2, 0.2, 0, 0, 1),
    (37, 640, 3, 16, 16, 0.1, 0, 0, 0),
    (65, 1024, 6, 32, 8, 0.1, 0, 0, 8),
    (129, 2304, 6, 384, 96, 0.1, 0, 0, 96),
    (64, 1152, 5, 8, 8, 0.0, 1, 16, 0),           # slots claimed, some dropped
    (300, 5120, 2, 12, 3, 0.5, 1, 64, 3),
    (517, 256, 7, 64, 64, 0.0, 0, 0, 0),
    (40, 512, 8, 32, 32, 1.0, 0, 0, 0),           # every slot padded
]


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("case", CASES)
def test_rows(case, dt):
    T, H, K, E, local, pad, mode, cap, begin = case
    say("rows", case, dt)
    s, d, w, R, g = make(T, H, K, E, local, pad, mode, cap, seed=T, begin=begin)
    slot, row = ref.route_rows(d.route_row, T, K, R)
    tok = torch.div(slot, K, rounding_mode="floor")
    # out: a copy; rows of no route keep what they held
    x = randn(g, (T, H), dt)
    rows = torch.full((R, H), 7.0, dtype=dt, device=DEV)
    moe.moe_permute(s, x, d.route_row, rows)
    want = torch.full((R, H), 7.0, dtype=dt)
    want[row] = x.cpu()[tok]
    assert torch.equal(rows.cpu(), want)
    # back: rows of no route hold NaN, which must not be read
    y = torch.full((R, H), float("nan"), dtype=dt)
    y[row] = torch.randn(len(row), H, generator=g).to(dt)
    y = y.to(DEV)
    for wt in (w, None):
        out = torch.full((T, H), 7.0, dtype=dt, device=DEV)
        moe.moe_unpermute(s, y, wt, d.route_row, out)
        o, mag = ref.unpermute(y, wt, d.route_row, T, K)
        # K products and K additions
        ref.assert_close(out, o, (K + 1) * ref.U32 * mag, "unpermute")
        if wt is None:
            dx = torch.full((T, H), 7.0, dtype=dt, device=DEV)
            moe.moe_permute_backward(s, y, d.route_row, dx)
            assert torch.equal(dx, out)
        elif dt is BF:
            old = torch.empty_like(out)
            moe.moe_combine(s, w, d.route_row, y, old)
            assert torch.equal(old.view(torch.int16), out.view(torch.int16))
    # gradients of the way back
    dout = randn(g, (T, H), dt)
    for wt in (w, None):
        drows = torch.full((R, H), 7.0, dtype=dt, device=DEV)
        dw = torch.full((T, K), 7.0, device=DEV)
        moe.moe_unpermute_backward(s, dout, y, wt, d.route_row, drows, dw)
        g64, y64 = dout.cpu().double()[tok], y.cpu().double()[row]
        ref_rows = torch.full((R, H), 7.0, dtype=torch.float64)
        ref_rows[row] = g64 if wt is None else g64 * w.cpu().double().reshape(-1)[slot][:, None]
        ref.assert_close(drows, ref_rows, ref.U32 * ref_rows.abs() * (wt is not None), "drows")
        ref_w, mag = torch.zeros(T * K).double(), torch.zeros(T * K).double()
        ref_w[slot], mag[slot] = (g64 * y64).sum(1), (g64 * y64).abs().sum(1)
        # a sum of H products in float32, in any order
        ref.assert_close(dw, ref_w.reshape(T, K), (H + 1) * ref.U32 * mag.reshape(T, K), "dw")
        # either one alone
        one, other = torch.full_like(drows, 7.0), torch.full_like(dw, 7.0)
        moe.moe_unpermute_backward(s, dout, None, wt, d.route_row, one, None)
        moe.moe_unpermute_backward(s, dout, y, wt, d.route_row, None, other)
        assert torch.equal(one, drows) and torch.equal(other, dw)


def test_no_tokens():
    s = moe.MoeShape(T=0, H=128, I=128, K=2, E_total=4, E_local=4)
    d = moe.alloc_dispatch(s, DEV)
    x = torch.empty(0, 128, dtype=BF, device=DEV)
    rows = torch.full((1, 128), 7.0, dtype=BF, device=DEV)
    w = torch.empty(0, 2, device=DEV)
    moe.moe_permute(s, x, d.route_row, rows)
    moe.moe_unpermute(s, rows, w, d.route_row, x)
    moe.moe_unpermute_backward(s, x, rows, w, d.route_row, rows, w)
    assert bool((rows == 7.0).all())


def test_indexes_past_the_rows_are_not_followed():
    s = moe.MoeShape(T=3, H=128, I=128, K=2, E_total=4, E_local=4)
    rr = torch.tensor([0, 6, 1 << 30, -2, -(1 << 31), 5], dtype=torch.int32, device=DEV)
    x = torch.randn(3, 128, device=DEV).to(BF)
    rows = torch.zeros(6, 128, dtype=BF, device=DEV)
    moe.moe_permute(s, x, rr, rows)
    want = torch.zeros_like(rows)
    want[0], want[5] = x[0], x[2]
    assert torch.equal(rows, want)
    out = torch.empty_like(x)
    moe.moe_unpermute(s, rows, None, rr, out)
    assert torch.equal(out, torch.stack([x[0], torch.zeros_like(x[0]), x[2]]))
    dw = torch.empty(3, 2, device=DEV)
    moe.moe_unpermute_backward(s, x, rows, None, rr, rows, dw)
    assert dw.cpu()[1].tolist() == [0.0, 0.0] and float(dw[0, 1]) == 0.0


def test_rows_past_32_bit_offsets():
    """Rows whose bytes lie past 2^32, every slot's row checked on the GPU."""
    T, H, K = 45000, 7168, 8
    s = moe.MoeShape(T=T, H=H, I=128, K=K, E_total=8, E_local=8)
    R = moe.moe_row_capacity(s)
    assert R * H * 2 > 1 << 32
    rr = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=DEV)   # the last rows first
    x = torch.randn(T, H, device=DEV).to(BF)
    rows = torch.zeros(R, H, dtype=BF, device=DEV)
    moe.moe_permute(s, x, rr, rows)
    flipped = rows.flip(0).reshape(T, K, H)
    for k in range(K):
        assert torch.equal(flipped[:, k], x)
    w = torch.full((T, K), 0.125, device=DEV)
    out = torch.empty_like(x)
    moe.moe_unpermute(s, rows, w, rr, out)
    assert torch.equal(out, x)                     # eight exact eighths
    dw = torch.empty_like(w)
    moe.moe_unpermute_backward(s, x, rows, w, rr, rows.zero_().add_(1), dw)
    assert torch.equal(rows.flip(0).reshape(T, K, H)[:, 3], (x.float() / 8).to(BF))


def test_streams_graphs_and_repeats():
    s, d, w, R, g = make(200, 1152, 6, 48, 24, 0.1, seed=4)
    w = torch.nan_to_num(w)
    x, y = randn(g, (200, 1152), BF), randn(g, (R, 1152), BF)
    rows, drows = torch.zeros_like(y), torch.zeros_like(y)
    dx, out = torch.empty_like(x), torch.empty_like(x)
    dw = torch.empty(200, 6, device=DEV)

    def step(stream=None):
        moe.moe_permute(s, x, d.route_row, rows, stream=stream)
        moe.moe_permute_backward(s, y, d.route_row, dx, stream=stream)
        moe.moe_unpermute(s, y, w, d.route_row, out, stream=stream)
        moe.moe_unpermute_backward(s, x, y, w, d.route_row, drows, dw, stream=stream)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (rows, dx, out, drows, dw)]

    step()
    first = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    assert all(torch.equal(a, b) for a, b in zip(results(), first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.normal_()
        y.normal_()
        step()
        eager = results()
        for t in (rows, dx, out, drows, dw):
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), eager))
