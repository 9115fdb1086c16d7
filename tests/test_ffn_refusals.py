"""The feed-forward block and the residual joint refuse bad shapes, types, pointers,
workspaces and tensors before any launch (no GPU is touched); and the gradients that the
kernels are tested against are those of the definitions, by differences."""

import ctypes
import math

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ffn_ref
from dispatch_grouped_gemm_amd import _build

FF = dict(T=16, H=512, I=256)
NO = dict(T=16, H=512)
FAKE, ODD = ctypes.c_void_p(256), ctypes.c_void_p(256 + 4)


@pytest.fixture(scope="module")
def lib():
    _build.build(force=False)
    return moe.lib()


def f_shape(**kw):
    return ctypes.byref(moe.FfnShape(**{**FF, **kw}).c())


def n_shape(**kw):
    return ctypes.byref(moe.NormShape(**{**NO, **kw}).c())


def test_shapes(lib):
    assert moe.moe_ffn_check(moe.FfnShape(**FF)) == 0
    assert moe.moe_ffn_check(moe.FfnShape(**FF, gate_limit=math.inf, up_limit=math.inf)) == 0
    for kw, code in [({"T": -1}, -1), ({"H": 0}, -1), ({"I": 0}, -1), ({"gate_limit": 0.0}, -1),
                     ({"gate_limit": math.nan}, -1), ({"up_limit": -1.0}, -1), ({"H": 48}, -2),
                     ({"I": 16}, -2), ({"H": (1 << 17) + 32}, -2), ({"I": (1 << 17) + 32}, -2),
                     ({"T": (1 << 24) + 1}, -2)]:
        s = moe.FfnShape(**{**FF, **kw})
        assert moe.moe_ffn_check(s) == code, kw
        assert moe.moe_ffn_workspace_size(s) == moe.moe_ffn_workspace_size(s, True) == 0
        c = ctypes.byref(s.c())
        assert lib.moe_ffn_forward(c, 0, *([FAKE] * 8), 1 << 40, None) == code
        assert lib.moe_ffn_backward(c, 0, *([FAKE] * 10), 0, 0, FAKE, 1 << 40, None) == code
    assert lib.moe_ffn_check(None) == lib.moe_norm_check(None) == -1
    assert moe.moe_ffn_workspace_size(moe.FfnShape(**{**FF, "T": 0}), True) == 0
    assert (moe.moe_ffn_workspace_size(moe.FfnShape(**FF), True)
            >= moe.moe_ffn_workspace_size(moe.FfnShape(**FF)) >= 16 * 256 * 2)
    assert moe.moe_norm_check(moe.NormShape(**NO, eps=0.0, skip_scale=-2.0)) == 0
    for kw, code in [({"T": -1}, -1), ({"H": 0}, -1), ({"eps": -1.0}, -1), ({"eps": math.nan}, -1),
                     ({"skip_scale": math.inf}, -1), ({"block_scale": math.nan}, -1),
                     ({"H": 40}, -2), ({"H": (1 << 14) + 32}, -2), ({"T": (1 << 24) + 1}, -2)]:
        s = moe.NormShape(**{**NO, **kw})
        assert moe.moe_norm_check(s) == code, kw
        assert moe.moe_norm_workspace_size(s) == 0
        c = ctypes.byref(s.c())
        assert lib.moe_norm_forward(c, 0, *([FAKE] * 9), None) == code
        assert lib.moe_norm_backward(c, 0, *([FAKE] * 13), 1 << 40, None) == code
    for word in ("feed-forward", "norms"):
        assert word in moe.moe_strerror(-2)


def test_ffn_forward_refusals(lib):
    f, ok = lib.moe_ffn_forward, f_shape()

    def args(**kw):
        v = dict(x=FAKE, w13=FAKE, w2=FAKE, base=FAKE, gu=FAKE, gs=FAKE, out=FAKE, ws=FAKE,
                 n=1 << 30)
        v.update(kw)
        return [*v.values(), None]

    for dt in (2, 3, -1):
        assert f(ok, dt, *args()) == -1
    for name in ("x", "w13", "w2", "out"):
        assert f(ok, 0, *args(**{name: None})) == -1, name
    for name in ("x", "w13", "w2", "base", "gu", "out"):
        assert f(ok, 0, *args(**{name: ODD})) == -1, name
    assert f(ok, 0, *args(gu=None)) == -1                 # exponents without codes
    assert f(ok, 0, *args(ws=None)) == -3
    assert f(ok, 0, *args(n=16)) == -3
    assert f(ok, 0, *args(ws=ctypes.c_void_p(256 + 16))) == -3
    assert f(f_shape(T=0), 0, *args(x=None, w13=None, out=None, ws=None)) == 0


def test_ffn_backward_refusals(lib):
    f, ok = lib.moe_ffn_backward, f_shape()

    def args(**kw):
        v = dict(dout=FAKE, x=FAKE, xs=None, w13=FAKE, w2=FAKE, gu=FAKE, gs=None, dx=FAKE,
                 dw13=FAKE, dw2=FAKE, dt=0, acc=0, ws=FAKE, n=1 << 30)
        v.update(kw)
        return [*v.values(), None]

    assert f(ok, 2, *args(dt=2)) == -1
    assert f(ok, 0, *args(dt=1)) == -1                    # neither dtype nor float32
    for name in ("dout", "x", "w13", "w2", "gu"):
        assert f(ok, 0, *args(**{name: None})) == -1, name
    for name in ("dout", "x", "w13", "w2", "gu", "dx", "dw13", "dw2"):
        assert f(ok, 0, *args(**{name: ODD})) == -1, name
    assert f(ok, 0, *args(x=None, xs=FAKE, dw13=None)) == -1
    assert f(ok, 0, *args(dx=None, dw13=None, dw2=None)) == -1
    assert f(ok, 0, *args(ws=None)) == -3
    assert f(ok, 0, *args(n=4096)) == -3
    assert f(f_shape(T=0), 0, *args(dout=None, dw13=None, dw2=None)) == 0


def test_norm_refusals(lib):
    f, ok = lib.moe_norm_forward, n_shape()

    def args(**kw):
        v = dict(x=FAKE, y=FAKE, w_post=FAKE, gate=FAKE, w_pre=FAKE, res=FAKE, normed=FAKE,
                 codes=None, exps=None)
        v.update(kw)
        return [*v.values(), None]

    assert f(ok, 3, *args()) == -1
    for kw in (dict(x=None), dict(y=None), dict(w_pre=None), dict(normed=None),
               dict(codes=FAKE), dict(exps=FAKE), dict(y=None, w_post=None, res=None),
               dict(y=None, gate=None, res=None), dict(y=None, w_post=None, gate=None),
               dict(res=None, w_pre=None, normed=None)):
        assert f(ok, 0, *args(**kw)) == -1, kw
    for name in ("x", "y", "w_post", "w_pre", "res", "normed"):
        assert f(ok, 0, *args(**{name: ODD})) == -1, name
    assert f(n_shape(T=0), 0, *args(x=None)) == 0

    b = lib.moe_norm_backward

    def back(**kw):
        v = dict(dn=FAKE, dres=FAKE, res=FAKE, y=FAKE, w_post=FAKE, gate=FAKE, w_pre=FAKE,
                 dx=FAKE, dy=FAKE, dgate=FAKE, dw_post=FAKE, dw_pre=FAKE, ws=FAKE, n=1 << 30)
        v.update(kw)
        return [*v.values(), None]

    assert b(ok, 3, *back()) == -1
    for kw in (dict(dn=None, dres=None, res=None, w_pre=None, dw_pre=None), dict(dn=None),
               dict(res=None), dict(w_pre=None), dict(dn=None, res=None, w_pre=None),
               dict(y=None), dict(w_post=None), dict(gate=None),
               dict(y=None, w_post=None, gate=None, dgate=None, dw_post=None),
               dict(dx=None, dy=None, dgate=None, dw_post=None, dw_pre=None)):
        assert b(ok, 0, *back(**kw)) == -1, kw
    for name in ("dn", "dres", "res", "y", "w_post", "w_pre", "dx", "dy"):
        assert b(ok, 0, *back(**{name: ODD})) == -1, name
    assert b(ok, 0, *back(ws=None)) == -3
    assert b(ok, 0, *back(n=256)) == -3


def test_binding_refuses_tensors(lib):
    """Wrong type, wrong shape, not contiguous, not on a GPU: refused in Python."""
    s = moe.FfnShape(T=4, H=64, I=32)
    x, bf = torch.zeros(4, 64, dtype=torch.bfloat16), torch.bfloat16
    w13, w2 = torch.zeros(64, 64, dtype=bf), torch.zeros(64, 32, dtype=bf)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.moe_ffn_forward(s, x, w13, w2, x, ws)         # host tensors
    with pytest.raises(TypeError):
        moe.moe_ffn_forward(s, x.float(), w13, w2, x, ws)
    with pytest.raises(TypeError):
        moe.moe_ffn_backward(s, None, x, w13, w2, x, x, w13, w2, ws)
    with pytest.raises(ValueError):
        moe.moe_ffn_backward(s, x, x, w13, w2, x, None, None, None, ws)
    n = moe.NormShape(T=4, H=64)
    with pytest.raises(ValueError):
        moe.moe_norm_forward(n, x, w2[0], x)
    with pytest.raises(TypeError):
        moe.moe_norm_backward(n, None, None, None, x, None, None)
    with pytest.raises(TypeError):
        moe.moe_norm_forward(n, x.double(), w2[0], x)


# ---- the reference's gradients ----------------------------------------------------------


def _difference(f, v, direction, eps=1e-6):
    return (f(v + eps * direction) - f(v - eps * direction)) / (2 * eps)


def test_ffn_reference_by_differences():
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, H, I, gl, ul = 5, 32, 32, 0.9, 1.1
    x, w13, w2, dout = n(T, H), n(2 * I, H) * 0.3, n(H, I), n(T, H)
    gu = x @ w13.t()

    def loss(x, w13, w2):
        a = x @ w13.t()
        h = ffn_ref.silu(ffn_ref.below(a[:, :I], gl)) * ffn_ref.cut(a[:, I:], ul)
        return (dout * (h @ w2.t())).sum()

    dx, _, dw13, _, dw2, _ = ffn_ref.ffn_backward(dout, x, w13, w2, gu, gl, ul, torch.float32)
    for grad, at in ((dx, 0), (dw13, 1), (dw2, 2)):
        args = [x, w13, w2]
        e = n(*args[at].shape)
        num = _difference(lambda v: loss(*args[:at], v, *args[at + 1:]), args[at], e)
        assert abs(float((grad * e).sum() - num)) <= 1e-6 * (1 + abs(float(num))), at


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_reference_by_differences(post, gated):
    g = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, H, eps, skip, scale = 4, 32, 1e-3, 1.5, 0.4
    v = dict(x=n(T, H), w_pre=n(H), y=n(T, H))
    if post:
        v["w_post"] = n(H)
    if gated:
        v["gate"] = n(T)
    dn, dres = n(T, H), n(T, H)

    def loss(v):
        r, _ = ffn_ref.norm_forward(v["x"], None, eps, skip, scale, v["y"], v.get("w_post"),
                                    v.get("gate"))
        return (dres * r).sum() + (dn * ffn_ref.norm_of(r, v["w_pre"], eps)[0]).sum()

    res, _ = ffn_ref.norm_forward(v["x"], None, eps, skip, scale, v["y"], v.get("w_post"),
                                  v.get("gate"))
    grads = ffn_ref.norm_backward(dn, dres, res, v["w_pre"], eps, skip, scale, v["y"],
                                  v.get("w_post"), v.get("gate"))
    for name in v:
        e = n(*v[name].shape)
        num = _difference(lambda t: loss({**v, name: t}), v[name], e)
        got = float((grads["d" + name][0] * e).sum())
        assert abs(got - float(num)) <= 1e-6 * (1 + abs(float(num))), name


def test_mx_reference_rounds_as_the_type():
    """The 64-bit 1x32 rule against torch's own conversion of scaled values."""
    g = torch.Generator().manual_seed(5)
    v = torch.randn(64, 96, generator=g).bfloat16() * torch.exp2(
        torch.randint(-9, 9, (64, 1), generator=g).float())
    codes, scale = ffn_ref.mx_rows(v)
    back = ffn_ref.mx_values(codes, scale)
    top = v.double().reshape(64, 3, 32).abs().amax(2, keepdim=True).expand(64, 3, 32).reshape(64, 96)
    # a step is at most 2^-3 of the value's binade or 2^-17 of the block's; the largest values
    # of a block may be cut from below 2^9 to 448 steps of its power
    allowed = torch.maximum(v.double().abs() * 2.0 ** -4, top * 2.0 ** -17)
    cutoff = v.double().abs() > top * 0.875
    assert ((back - v.double()).abs() <= torch.where(cutoff, top * 0.125, allowed)).all()
