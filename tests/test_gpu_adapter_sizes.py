"""The adapters at sizes for both forms of few rows of a given projection and for every
kernel of many rows: the shrinks of 16 x 16, 32 x 32 and
32 x 64 over many steps, the tiles of every kind over many steps (their rings refilled
many times), ranks that take several turns, several adapters in every 16 rows.

Which kernels a size reaches is said for 256 CUs."""

import pytest
import torch

import ops_ref as ref
from gpu_util import DEV, say
from test_gpu_adapter import ids_of, project, whole

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16

SIZES = [
    # T, H, N, L, rank
    (40, 1024, 72, 5, 128),                        # few rows; given projections in any order,
    (41, 1024, 72, 5, 128),                        # and by adapter
    (64, 2048, 392, 30, 64),
    (128, 4096, 2104, 9, 48),                      # few rows by 128 columns
    (4111, 2304, 264, 13, 128),                    # shrink by 32 x 64; tiles in parts of H
    (4111, 1152, 392, 300, 40),                    # shrink by 32 x 32, most blocks not full
    (8191, 768, 520, 5, 24),                       # the same; two workgroups a CU
    (8191, 1280, 264, 40, 64),                     # 32 x 64
    (9000, 640, 136, 21, 72),                      # 32 x 64, two walks of the order
    (300, 2048, 520, 90, 136),                     # 16 x 16; eight parts
    (520, 4224, 4480, 6, 72),                      # two parts of 175 tiles
    (400, 4224, 6152, 11, 40),                     # one deep workgroup a CU (196 tiles)
    (256, 2304, 11000, 60, 256),                   # the same (172 tiles)
    (700, 1152, 4352, 200, 256),                   # two workgroups a CU (204 tiles)
    (1300, 1152, 4096, 30, 72),                    # the same (352 tiles)
    (4111, 1152, 4504, 17, 72),                    # 256 x 256: 306 tiles, 50 as halves
    (4111, 896, 6104, 400, 16),                    # 408 tiles, none halved
]


def terms(x, w, base, ids, a, b, scale):
    """out in 64 bits, and the bound on the float32 sums' error: sums of H products, then of
    the 3 rank (bf16) or 6 rank (fp16) products of the parts of v and B, which have one
    sign and add up to v and B; each sum of n terms off by at most (n + 2) 2^-24 of the
    terms' magnitudes, the scale and the last addition by 2^-24 each."""
    x, a, b = x.cpu().double(), a.cpu().double(), b.cpu().double()
    H, r = x.shape[1], a.shape[1]
    if w is None:
        out = base.cpu().double()
        off = torch.zeros_like(out)
    else:
        w = w.cpu().double()
        out = x @ w.t()
        off = (H + 2) * ref.U32 * (x.abs() @ w.abs().t())
    for l in range(a.shape[0]):
        at = torch.nonzero(ids.cpu() == l)[:, 0]
        if not at.numel():
            continue
        s, bt = 1.0 if scale is None else float(scale[l]), b[l].t()
        v = x[at] @ a[l].t()
        v_off = (H + 2) * ref.U32 * (x[at].abs() @ a[l].abs().t())
        out[at] += s * (v @ bt)
        off[at] += s * ((v_off + (6 * r + 4) * ref.U32 * (v.abs() + v_off)) @ bt.abs())
    return out, off + ref.U32 * (out.abs() + off)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("size", SIZES)
def test_whole_numbers(size, dt):
    """As at the smaller sizes: 2 H rank times the largest scale, 4, is below 2^24, so every
    sum is exact in float32 and the output the exact value rounded once."""
    T, H, N, L, r = size
    assert 8 * H * r + 2 * H < 1 << 24
    g = torch.Generator().manual_seed(T * 11 + H)
    x = whole(g, (T, H), -2, 2, dt)
    x[:, torch.rand(H, generator=g).to(DEV) < 0.5] = 0
    w = whole(g, (N, H), -1, 1, dt)
    a, b = whole(g, (L, r, H), -1, 1, dt), whole(g, (L, N, r), -1, 1, dt)
    scale = (2.0 ** torch.randint(-1, 3, (L,), generator=g)).to(DEV)
    base = whole(g, (T, N), -50, 50, dt)
    for kind, ww, bb in (("mixed", w, None), ("requests", w, None), ("requests", None, base),
                         ("mixed", None, base)):
        ids = ids_of(kind, T, L, g).to(DEV)
        say("adapter sizes", size, dt, kind, ww is not None)
        out = project(T, H, N, L, r, dt, x, ww, bb, ids, a, b, scale)
        want, _ = terms(x, ww, bb, ids, a, b, scale)
        assert torch.equal(out.cpu(), want.to(dt)), (kind, ww is not None)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("size", SIZES)
def test_normal_numbers(size, dt):
    T, H, N, L, r = size
    g = torch.Generator().manual_seed(T * 5 + H)
    rn = lambda shape, std: (torch.randn(shape, generator=g) * std).to(dt).to(DEV)
    x, w = rn((T, H), 1.0), rn((N, H), H ** -0.5)
    a, b = rn((L, r, H), H ** -0.5), rn((L, N, r), r ** -0.5)
    scale, base = torch.rand(L, generator=g).to(DEV) * 2, rn((T, N), 1.0)
    for kind, ww, bb in (("mixed", w, None), ("requests", None, base)):
        ids = ids_of(kind, T, L, g).to(DEV)
        say("adapter sizes", size, dt, kind, ww is not None)
        out = project(T, H, N, L, r, dt, x, ww, bb, ids, a, b, scale)
        want, off = terms(x, ww, bb, ids, a, b, scale)
        ref.assert_close(out, want, off, str(size))
