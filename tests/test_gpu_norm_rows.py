"""Many short rows: several to a workgroup in the joint's gradients, the last set not full; the
same call twice gives the same bits; rows beside each other do not see one another."""

import math

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ffn_ref
import test_gpu_norm as base
from ops_ref import assert_close

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("T,H", [(513, 32), (700, 96), (1500, 544), (4099, 160), (5001, 512),
                                 (1027, 1312), (2050, 2080), (1100, 4128)])
def test_gradients(T, H, dt):
    for y, post, gated in ((True, True, True), (True, False, True), (False, False, False)):
        c = base._case(T, H, dt, T + H, y, post, gated)
        s = moe.NormShape(T=T, H=H, eps=1e-5, skip_scale=0.75, block_scale=0.4)
        ws = moe.alloc_norm_workspace(s, DEV)
        res = c["x"]
        kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
        first = None
        for _ in range(2):
            o = dict(dx=torch.full((T + 1, H), -3.0, dtype=dt, device=DEV),
                     dw_pre=torch.full((H,), 9.0, device=DEV))
            if y:
                o["dy"] = torch.full((T + 1, H), -3.0, dtype=dt, device=DEV)
            if post:
                o["dw_post"] = torch.full((H,), 9.0, device=DEV)
            if gated:
                o["dgate"] = torch.full((T + 1,), 9.0, device=DEV)
            ws.fill_(255)
            moe.moe_norm_backward(s, c["dnormed"], res, c["w_pre"], o["dx"][:T], o["dw_pre"], ws,
                                  dres=c["dres"], dy=o["dy"][:T] if y else None,
                                  dw_post=o.get("dw_post"),
                                  dgate=o["dgate"][:T] if gated else None, **kw)
            assert first is None or all(torch.equal(first[k], o[k]) for k in o)
            first = o
        r = ffn_ref.norm_backward(c["dnormed"], c["dres"], res, c["w_pre"], 1e-5, 0.75, 0.4, **kw)
        for k, (v, b) in r.items():
            assert_close(o[k][:T] if k in ("dx", "dy", "dgate") else o[k], v, b, k)
        for k in ("dx", "dy"):
            assert k not in o or (o[k][T] == -3).all()
        assert not gated or o["dgate"][T] == 9


def test_rows_of_a_workgroup_are_apart():
    """A row of NaN among rows that share its workgroup: their gradients keep their bits."""
    T, H = 3000, 96
    c = base._case(T, H, BF, 3)
    s = moe.NormShape(T=T, H=H)
    kw = dict(y=c["y"], w_post=c["w_post"], gate=c["gate"])
    out = []
    for bad in (False, True):
        res = c["x"].clone()
        if bad:
            res[1234, 5] = math.nan
        dx, dy, dg = torch.empty_like(res), torch.empty_like(res), torch.empty(T, device=DEV)
        moe.moe_norm_backward(s, c["dnormed"], res, c["w_pre"], dx, None, None, dres=c["dres"],
                              dy=dy, dgate=dg, **kw)
        out.append((dx, dy, dg))
    rest = torch.arange(T, device=DEV) != 1234
    for a, b in zip(*out):
        assert torch.equal(a[rest], b[rest]) and b[1234].isnan().all()
