"""The feed-forward block at sizes for each of its tiles, whole and with K in parts, and for the
cuts of a last round; what is not finite in 8 bits; and workspaces that hold anything."""

import math

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ffn_ref
import test_gpu_ffn as base
from ops_ref import assert_close

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16
DEV = "cuda"

# rows by H by I; first product, second product, dh
SIZES = [(8278, 448, 256),      # 128 x 256, 128 x 256, 128 x 128
         (11648, 128, 1024),    # 256 x 256 with halves left over
         (4937, 4672, 2656),    # 256 x 256 with quarters, with halves
         (1021, 2304, 1408),    # 128 x 128 both, 64 x 128
         (85, 4032, 2848),      # 128 x 128 in parts
         (69, 6048, 2016),      # 64 x 128 in parts, dh too
         (816, 1280, 4064),     # second product 128 x 128 in parts
         (155, 1504, 3712),     # second product 64 x 128 in parts
         (216, 448, 2048),      # second product 32 x 64 in parts
         (789, 4000, 96),       # second product 128 x 128, dh 64 x 64 in parts
         (167, 3168, 128),      # second product 64 x 64
         (4694, 160, 800),      # dh 128 x 256
         (13548, 544, 1600),    # dh 256 x 256 with halves left over
         (214, 7168, 2112),     # dh 128 x 128 in parts
         (8420, 192, 128),      # dh 64 x 128
         (14, 6304, 608),       # few rows of a long K: tiles in parts, then 32 columns
         (40, 480, 1568), (50, 2400, 1024), (64, 5120, 2304)]  # up to 64 rows, 32 columns


@pytest.mark.parametrize("T,H,I", SIZES)
def test_forward_whole_numbers(T, H, I):
    base.test_forward_whole_numbers(T, H, I, F16 if T % 2 else BF)


@pytest.mark.parametrize("T,H,I", SIZES)
def test_backward_whole_numbers(T, H, I):
    base.test_backward_whole_numbers(T, H, I, BF if T % 2 else F16)


@pytest.mark.parametrize("T", [1, 16, 40, 64, 65, 300])
def test_not_finite_in_8_bits(T):
    """Infinities and NaN of g and u are kept as NaN, the block's other values by the exponent
    that they have without them; the gradients of that row are NaN, of no other."""
    H, I = 288, 160
    g = base._gen(T)
    s = moe.FfnShape(T=T, H=H, I=I, gate_limit=math.inf, up_limit=math.inf)
    ws = moe.alloc_ffn_workspace(s, DEV, backward=True)
    x = base._ints(g, -2, 2, T, H).to(BF)
    w13 = base._ints(g, -1, 1, 2 * I, H).to(BF)
    w2 = base._normal(g, BF, 0.1, H, I)
    row = T // 2
    w13[3] = 0
    w13[3, 0], x[row, 0], x[[t for t in range(T) if t != row], 0] = math.inf, 1, 0
    gu = x.double() @ torch.where(w13.isinf(), 0.0, w13.double()).t()
    codes = torch.empty(T, 2 * I, dtype=torch.uint8, device=DEV)
    exps = torch.empty(T, 2 * I // 32, dtype=torch.uint8, device=DEV)
    moe.moe_ffn_forward(s, x, w13, w2, torch.empty_like(x), ws, gate_up=codes, gate_up_scale=exps)
    gu[:, 3] = 0
    c, e = ffn_ref.mx_rows(gu)
    got = codes.cpu()
    # 0 times infinity: NaN in every other row's column 3, infinity in `row`
    assert ((got[:, 3] & 0x7f) == 0x7f).all()
    c[:, 3] = got[:, 3]
    zero = (c & 0x7f) == 0
    assert torch.equal(exps.cpu(), e)
    assert torch.equal(torch.where(zero, got & 0x7f, got), torch.where(zero, 0, c))
    # gradients: only the rows that hold one are NaN
    codes2 = codes.clone()
    codes2[:, 3] = torch.where(torch.arange(T, device=DEV) == row, 0x7f, 0).to(torch.uint8)
    dx = torch.empty_like(x)
    w13[3] = 1
    moe.moe_ffn_backward(s, base._normal(g, BF, 1, T, H), None, w13, w2, codes2, dx, None, None, ws,
                         gate_up_scale=exps)
    nan = dx.isnan().all(1)
    assert bool(nan[row]) and int(nan.sum()) == 1 and int(dx.isnan().any(1).sum()) == 1


@pytest.mark.parametrize("T,H,I", [(3, 96, 64), (64, 2304, 96), (100, 1024, 512), (300, 1632, 352)])
def test_workspace_holds_anything(T, H, I):
    """NaN in the workspace beforehand, a larger one than asked for, the smallest one."""
    g = base._gen(7)
    x, w13 = base._normal(g, BF, 1, T, H), base._normal(g, BF, 0.05, 2 * I, H)
    w2, dout = base._normal(g, BF, 0.1, H, I), base._normal(g, BF, 1, T, H)
    s = moe.FfnShape(T=T, H=H, I=I)
    results = []
    for more in (0, 4096):
        n = moe.moe_ffn_workspace_size(s, True) + more
        ws = torch.full((n + 512,), 255, dtype=torch.uint8, device=DEV)
        kept = torch.empty(T, 2 * I, dtype=BF, device=DEV)
        out, dx = torch.empty_like(x), torch.empty_like(x)
        dw13, dw2 = torch.empty_like(w13), torch.empty_like(w2)
        moe.moe_ffn_forward(s, x, w13, w2, out, ws[:n], gate_up=kept)
        moe.moe_ffn_backward(s, dout, x, w13, w2, kept, dx, dw13, dw2, ws[:n])
        assert (ws[n:] == 255).all()
        results.append((out, kept, dx, dw13, dw2))
    for a, b in zip(*results):
        assert torch.equal(a, b) and not a.isnan().any()
    with pytest.raises(moe.MoeError):
        moe.moe_ffn_forward(s, x, w13, w2, out, ws[:moe.moe_ffn_workspace_size(s) - 256])


def test_a_block_as_it_is_used():
    """Norm, router, experts and the dense block added to them, the joint behind, and back: each
    step from what the step before gave, inside its own bounds."""
    T, H, I, K, E = 70, 512, 256, 2, 8
    g = base._gen(21)
    n = moe.NormShape(T=T, H=H, block_scale=0.5)
    f = moe.FfnShape(T=T, H=H, I=I)
    m = moe.MoeShape(T=T, H=H, I=I, K=K, E_total=E, E_local=E)
    x = base._normal(g, BF, 1, T, H)
    w_in, w_post, w_next = [(1 + base._normal(g, BF, 0.1, H)).to(BF) for _ in range(3)]
    gate = torch.randn(T, generator=g, device=DEV)
    w13, w2 = base._normal(g, BF, 1.5 * H ** -0.5, 2 * I, H), base._normal(g, BF, I ** -0.5, H, I)
    router = base._normal(g, BF, H ** -0.5, E, H)
    e13 = torch.randint(0, 256, (E, 2 * I, H // 2), generator=g, device=DEV, dtype=torch.uint8)
    e2 = torch.randint(0, 256, (E, H, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    s13 = torch.full((E, 2 * I, H // 32), 121, dtype=torch.uint8, device=DEV)
    s2 = torch.full((E, H, I // 32), 121, dtype=torch.uint8, device=DEV)
    # forward
    a, a8 = torch.empty_like(x), torch.empty(T, H, dtype=torch.uint8, device=DEV)
    a8s = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV)
    moe.moe_norm_forward(n, x, w_in, a, normed_fp8=a8, normed_scale=a8s)
    assert_close(a, *ffn_ref.norm_of(x, w_in, 1e-6), "normed")
    ids, w = torch.empty(T, K, dtype=torch.int32, device=DEV), torch.empty(T, K, device=DEV)
    moe.moe_route(m, (a.float() @ router.float().t()).to(BF), ids, w)
    experts = torch.empty_like(x)
    moe.moe_forward(m, a8, a8s, ids, w, e13, s13, e2, s2, experts, moe.alloc_workspace(m, DEV))
    ws = moe.alloc_ffn_workspace(f, DEV, backward=True)
    y = experts.clone()
    kept = torch.empty(T, 2 * I, dtype=torch.uint8, device=DEV)
    exps = torch.empty(T, 2 * I // 32, dtype=torch.uint8, device=DEV)
    moe.moe_ffn_forward(f, a, w13, w2, y, ws, base=y, gate_up=kept, gate_up_scale=exps)
    ref, off, _, _ = ffn_ref.ffn_forward(a, w13, w2, 10.0, 10.0, experts)
    assert_close(y, ref, off, "out")
    res, nxt = torch.empty_like(x), torch.empty_like(x)
    moe.moe_norm_forward(n, x, w_next, nxt, y=y, w_post=w_post, gate=gate, res=res)
    assert_close(res, *ffn_ref.norm_forward(x, None, 1e-6, 1.0, 0.5, y, w_post, gate), "res")
    assert_close(nxt, *ffn_ref.norm_of(res, w_next, 1e-6), "next")
    # back to x by way of the dense block
    dn, dr = base._normal(g, BF, 1, T, H), base._normal(g, BF, 1, T, H)
    nws = moe.alloc_norm_workspace(n, DEV)
    dskip, dy = torch.empty_like(x), torch.empty_like(x)
    dg, dwp, dwn = (torch.empty(T, device=DEV), torch.empty(H, device=DEV),
                    torch.empty(H, device=DEV))
    moe.moe_norm_backward(n, dn, res, w_next, dskip, dwn, nws, dres=dr, y=y, w_post=w_post,
                          gate=gate, dy=dy, dw_post=dwp, dgate=dg)
    r = ffn_ref.norm_backward(dn, dr, res, w_next, 1e-6, 1.0, 0.5, y, w_post, gate)
    for t, k in ((dskip, "dx"), (dy, "dy"), (dg, "dgate"), (dwp, "dw_post"), (dwn, "dw_pre")):
        assert_close(t, *r[k], k)
    da, dw13, dw2 = torch.empty_like(x), torch.zeros(2 * I, H, device=DEV), torch.zeros(H, I, device=DEV)
    moe.moe_ffn_backward(f, dy, a8, w13, w2, kept, da, dw13, dw2, ws, gate_up_scale=exps,
                         x_scale=a8s, accumulate=True)
    r = ffn_ref.ffn_backward(dy, ffn_ref.mx_values(a8, a8s).to(DEV), w13, w2,
                             ffn_ref.mx_values(kept, exps).to(DEV), 10.0, 10.0, BF)
    for i, t in enumerate((da, dw13, dw2)):
        assert_close(t, r[2 * i], r[2 * i + 1], "gradient %d" % i)
    dx = torch.empty_like(x)
    moe.moe_norm_backward(n, da, x, w_in, dx, None, None, dres=dskip)
    r = ffn_ref.norm_backward(da, dskip, x, w_in, 1e-6, 1.0, 0.5)
    assert_close(dx, *r["dx"], "dx")
