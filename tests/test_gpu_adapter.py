"""The shared projection with low-rank adapters against the 64-bit definition."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ops_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def ids_of(kind, T, L, g):
    if kind == "mixed":
        ids = torch.randint(-1, L, (T,), generator=g)
    elif kind == "requests":
        cuts = torch.sort(torch.randint(0, T + 1, (5,), generator=g)).values
        of = torch.randint(-1, L, (6,), generator=g)
        ids = of[(torch.arange(T)[:, None] >= cuts[None, :]).sum(1)]
    elif kind == "none":
        ids = torch.full((T,), -1)
    elif kind == "one":
        ids = torch.full((T,), L - 1)
    else:                                          # ids that name no adapter
        ids = torch.where(torch.arange(T) % 2 == 0, L + 5, -7)
        ids[T // 2] = 0
    return ids.to(torch.int32)


def project(T, H, N, L, r, dt, x, w, base, ids, a, b, scale, out=None):
    s = moe.AdapterShape(T=T, H=H, N=N, L=L, rank=r)
    ws = moe.alloc_adapter_workspace(s, DEV)
    ws.fill_(255)                                  # nothing in it needs clearing
    if out is None:
        out = torch.full((T, N), 7.0, dtype=dt, device=DEV)
    moe.moe_adapter_project(s, x, w, ids, a, b, scale, out, ws, base=base)
    return out


def whole(g, shape, lo, hi, dt):
    return torch.randint(lo, hi + 1, shape, generator=g).to(dt).to(DEV)


SIZES = [
    # T, H, N, L, rank
    (1, 128, 8, 1, 8),
    (1, 5120, 1536, 8, 16),
    (2, 256, 72, 3, 24),
    (15, 384, 200, 40, 8),
    (16, 128, 384, 2, 64),
    (17, 640, 64, 5, 40),
    (33, 512, 136, 3, 256),
    (64, 1024, 256, 64, 16),
    (65, 896, 520, 7, 32),
    (128, 2304, 640, 33, 128),
    (200, 512, 1000, 4, 16),
    (257, 1152, 264, 100, 8),
    (511, 768, 768, 6, 64),
    (700, 256, 2304, 3, 16),
    (1025, 384, 392, 12, 48),
    (130, 2048, 200, 6, 16),                       # parts of H by tiles
    (700, 1536, 3000, 20, 40),                     # no more tiles than CUs
    (1300, 256, 4100 - 4, 7, 8),                   # more
    (9000, 128, 40, 70, 8),                        # more rows than a batch of the order
    (9000, 128, 16, 9000, 8),                      # both
    (300, 128, 64, 9000, 8),                       # more adapters than the order counts in LDS
    (4111, 128, 4104, 9, 16),                      # the largest tiles
]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("size", SIZES)
def test_whole_numbers(size, dt):
    """Small whole numbers: every product and sum is exact in float32 (magnitudes below
    2^24, v below 2^15), so the output is the exact value rounded once: the same bits."""
    T, H, N, L, r = size
    g = torch.Generator().manual_seed(T * 7 + H)
    x = whole(g, (T, H), -2, 2, dt)
    x[:, torch.rand(H, generator=g).to(DEV) < 0.5] = 0
    w = whole(g, (N, H), -1, 1, dt)
    a, b = whole(g, (L, r, H), -1, 1, dt), whole(g, (L, N, r), -1, 1, dt)
    scale = (2.0 ** torch.randint(-1, 3, (L,), generator=g)).to(DEV)
    base = whole(g, (T, N), -50, 50, dt)
    for kind in ("mixed", "requests", "none", "one", "outside"):
        if T * L > 1 << 24 and kind != "mixed":
            continue                               # the reference walks the adapters
        ids = ids_of(kind, T, L, g).to(DEV)
        for ww, bb, sc in ((w, None, scale), (None, base, None)):
            say("adapter", size, dt, kind, ww is not None)
            out = project(T, H, N, L, r, dt, x, ww, bb, ids, a, b, sc)
            want, _ = ref.adapters(x, ww, bb, ids, a, b, sc)
            assert torch.equal(out.cpu(), want.to(dt)), (kind, ww is not None)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("size", SIZES)
def test_normal_numbers(size, dt):
    T, H, N, L, r = size
    g = torch.Generator().manual_seed(T * 3 + H)
    rn = lambda shape, std: (torch.randn(shape, generator=g) * std).to(dt).to(DEV)
    x, w = rn((T, H), 1.0), rn((N, H), H ** -0.5)
    a, b = rn((L, r, H), H ** -0.5), rn((L, N, r), r ** -0.5)
    scale, base = torch.rand(L, generator=g).to(DEV) * 2, rn((T, N), 1.0)
    for kind in ("mixed", "requests"):
        ids = ids_of(kind, T, L, g).to(DEV)
        for ww, bb in ((w, None), (None, base)):
            say("adapter", size, dt, kind, ww is not None)
            out = project(T, H, N, L, r, dt, x, ww, bb, ids, a, b, scale)
            want, off = ref.adapters(x, ww, bb, ids, a, b, scale)
            ref.assert_close(out, want, off, str(size))


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_half_range_and_large_products(T):
    """x A^T far outside fp16's range (about 2^20) and far below it (2^-20) comes back
    through B as the definition says."""
    H, N, L, r = 256, 264, 3, 16
    g = torch.Generator().manual_seed(8)
    x = (torch.randn(T, H, generator=g) * 256).to(HF).to(DEV)
    ids = ids_of("mixed", T, L, g).to(DEV)
    base = torch.zeros(T, N, dtype=HF, device=DEV)
    for up in (1.0, -1.0):
        a = (torch.randn(L, r, H, generator=g) * 2.0 ** (8 * up)).to(HF).to(DEV)
        xs = x if up > 0 else (x * 2.0 ** -18).to(HF)
        b = (torch.randn(L, N, r, generator=g) * 2.0 ** (-12 * up)).to(HF).to(DEV)
        out = project(T, H, N, L, r, HF, xs, None, base, ids, a, b, None)
        want, off = ref.adapters(xs, None, base, ids, a, b, None)
        ref.assert_close(out, want, off, "range")


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T", [5, 48, 300])
def test_one_adapter_never_reaches_anothers_rows(T, dt):
    """An adapter of infinities and NaN changes its own rows only; a row of NaN its own."""
    H, N, L, r = 256, 136, 4, 16
    g = torch.Generator().manual_seed(9)
    rn = lambda shape: torch.randn(shape, generator=g).to(dt).to(DEV)
    x, w, a, b = rn((T, H)), rn((N, H)), rn((L, r, H)) / 16, rn((L, N, r))
    ids = ids_of("mixed", T, L, g)
    ids[:3] = torch.tensor([0, 1, 2])
    ids = ids.to(DEV)
    good = project(T, H, N, L, r, dt, x, w, None, ids, a, b, None)
    a2, b2 = a.clone(), b.clone()
    a2[1], b2[1] = float("inf"), float("nan")
    b2[3] = float("inf")
    bad = project(T, H, N, L, r, dt, x, w, None, ids, a2, b2, None)
    keep = (ids != 1) & (ids != 3)
    assert torch.equal(bad[keep], good[keep])
    assert bool(torch.isnan(bad[ids == 1]).all())
    x2 = x.clone()
    x2[0] = float("nan")
    other = project(T, H, N, L, r, dt, x2, w, None, ids, a, b, None)
    assert torch.equal(other[1:], good[1:]) and bool(torch.isnan(other[0]).all())


def test_base_in_place_and_workspace_larger_than_needed():
    T, H, N, L, r = 77, 512, 392, 5, 16
    g = torch.Generator().manual_seed(10)
    rn = lambda shape, std=1.0: (torch.randn(shape, generator=g) * std).to(BF).to(DEV)
    x, a, b, base = rn((T, H)), rn((L, r, H), 0.05), rn((L, N, r)), rn((T, N))
    ids = ids_of("mixed", T, L, g).to(DEV)
    want = project(T, H, N, L, r, BF, x, None, base, ids, a, b, None)
    there = base.clone()
    project(T, H, N, L, r, BF, x, None, there, ids, a, b, None, out=there)
    assert torch.equal(there, want)
    assert torch.equal(want[ids < 0], base[ids < 0])


def test_rows_behind_the_last_are_left():
    """out, and what lies behind the workspace, are written to their ends and no further."""
    T, H, N, L, r = 19, 256, 72, 3, 24
    g = torch.Generator().manual_seed(11)
    rn = lambda shape: torch.randn(shape, generator=g).to(BF).to(DEV)
    x, w, a, b = rn((T, H)), rn((N, H)), rn((L, r, H)), rn((L, N, r))
    ids = ids_of("mixed", T, L, g).to(DEV)
    s = moe.AdapterShape(T=T, H=H, N=N, L=L, rank=r)
    need = moe.moe_adapter_workspace_size(s)
    ws = torch.full((need + 4096,), 91, dtype=torch.uint8, device=DEV)
    room = torch.full((T + 200, N), 7.0, dtype=BF, device=DEV)
    moe.moe_adapter_project(s, x, w, ids, a, b, None, room[:T], ws[:need])
    assert bool((room[T:] == 7.0).all()) and bool((ws[need:] == 91).all())


@pytest.mark.parametrize("T,H,N,L,r", [(1, 512, 640, 4, 16), (96, 1024, 512, 20, 32),
                                       (600, 512, 768, 5, 16)])
def test_streams_graphs_and_repeats(T, H, N, L, r):
    g = torch.Generator().manual_seed(12)
    rn = lambda shape, std=1.0: (torch.randn(shape, generator=g) * std).to(BF).to(DEV)
    x, w = rn((T, H)), rn((N, H), H ** -0.5)
    a, b = rn((L, r, H), H ** -0.5), rn((L, N, r))
    ids = ids_of("mixed", T, L, g).to(DEV)
    s = moe.AdapterShape(T=T, H=H, N=N, L=L, rank=r)
    ws = moe.alloc_adapter_workspace(s, DEV)
    out = torch.empty(T, N, dtype=BF, device=DEV)
    call = lambda st=None: moe.moe_adapter_project(s, x, w, ids, a, b, None, out, ws, stream=st)
    call()
    torch.cuda.synchronize()
    first = out.clone()
    for _ in range(4):                             # the same bits every time
        out.zero_()
        call()
        assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    call(side)
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        x.normal_()
        ids.copy_(torch.randint(-1, L, (T,), generator=g).to(torch.int32))
        call()
        torch.cuda.synchronize()
        eager = out.clone()
        out.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_a_large_weight():
    """Sizes where the weight passes 2^32 bytes, in whole numbers, sampled."""
    T, H, N, L, r = 3, 8192, 300000, 2, 8
    g = torch.Generator().manual_seed(13)
    x = whole(g, (T, H), -1, 1, BF)
    x[:, 64:] = 0
    w = torch.ones(N, H, dtype=BF, device=DEV)
    w[::2] = -1
    a, b = whole(g, (L, r, H), -1, 1, BF), whole(g, (L, N, r), -1, 1, BF)
    ids = torch.tensor([1, -1, 0], dtype=torch.int32, device=DEV)
    out = project(T, H, N, L, r, BF, x, w, None, ids, a, b, None)
    pick = torch.tensor([0, 1, 2, 777, 131071, 262144, 270001, 299998, 299999])
    want, _ = ref.adapters(x, w[pick.to(DEV)], None, ids, a, b[:, pick.to(DEV)], None)
    assert torch.equal(out[:, pick.to(DEV)].cpu(), want.to(BF))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T,N", [(65, 4744), (100, 4800), (128, 15000)])
def test_few_rows_of_a_wide_weight(T, N, dt):
    """A long H by many columns, whole numbers as above: exact in float32."""
    H, L, r = 4096, 5, 24
    g = torch.Generator().manual_seed(T)
    x = whole(g, (T, H), -2, 2, dt)
    x[:, torch.rand(H, generator=g).to(DEV) < 0.5] = 0
    w = whole(g, (N, H), -1, 1, dt)
    a, b = whole(g, (L, r, H), -1, 1, dt), whole(g, (L, N, r), -1, 1, dt)
    base = whole(g, (T, N), -50, 50, dt)
    for kind in ("mixed", "requests", "none", "one"):
        ids = ids_of(kind, T, L, g).to(DEV)
        for ww, bb in ((w, None), (None, base)):
            say("adapter wide", T, N, dt, kind, ww is not None)
            out = project(T, H, N, L, r, dt, x, ww, bb, ids, a, b, None)
            want, _ = ref.adapters(x, ww, bb, ids, a, b, None)
            assert torch.equal(out.cpu(), want.to(dt)), (kind, ww is not None)
