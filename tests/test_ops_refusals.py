"""The router, the rows to their experts and back, and the adapters refuse bad shapes,
types, pointers, workspaces and tensors before any launch (no GPU is touched)."""

import ctypes

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
from dispatch_grouped_gemm_amd import _build

V4 = dict(T=128, H=7168, I=512, K=6, E_total=384, E_local=48)
AD = dict(T=16, H=512, N=256, L=4, rank=16)
FAKE, ODD = ctypes.c_void_p(256), ctypes.c_void_p(256 + 4)


@pytest.fixture(scope="module")
def lib():
    _build.build(force=False)
    return moe.lib()


def c_shape(**kw):
    return ctypes.byref(moe.MoeShape(**{**V4, **kw}).c())


def a_shape(**kw):
    return ctypes.byref(moe.AdapterShape(**{**AD, **kw}).c())


def test_route_refusals(lib):
    ok = c_shape()
    assert lib.moe_route(c_shape(K=0), 0, FAKE, 1, FAKE, FAKE, None) == -1
    assert lib.moe_route(ok, 3, FAKE, 1, FAKE, FAKE, None) == -1
    assert lib.moe_route(ok, -1, FAKE, 1, FAKE, FAKE, None) == -1
    for i in (2, 4, 5):
        args = [ok, 0, FAKE, 1, FAKE, FAKE, None]
        args[i] = None
        assert lib.moe_route(*args) == -1
    assert lib.moe_route(c_shape(E_total=1025), 0, FAKE, 1, FAKE, FAKE, None) == -2
    assert lib.moe_route(c_shape(T=0), 0, None, 1, None, None, None) == 0
    for i in (4, 5, 6, 7):
        args = [ok, 0, FAKE, 1, FAKE, FAKE, FAKE, FAKE, None]
        args[i] = None
        assert lib.moe_route_backward(*args) == -1
    # the logits are needed for the softmax over all experts
    assert lib.moe_route_backward(ok, 0, None, 0, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert lib.moe_route_backward(ok, 7, FAKE, 1, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert lib.moe_route_backward(c_shape(E_total=2000), 0, FAKE, 1, FAKE, FAKE, FAKE, FAKE,
                                  None) == -2
    assert lib.moe_route_backward(c_shape(T=0), 0, None, 1, None, None, None, None, None) == 0


def test_row_refusals(lib):
    ok, z = c_shape(), c_shape(T=0)
    for fn in (lib.moe_permute, lib.moe_permute_backward):
        assert fn(c_shape(H=100), 0, FAKE, FAKE, FAKE, None) == -2
        assert fn(ok, 5, FAKE, FAKE, FAKE, None) == -1
        for i in (2, 3, 4):
            args = [ok, 0, FAKE, FAKE, FAKE, None]
            args[i] = None
            assert fn(*args) == -1
        assert fn(ok, 0, ODD, FAKE, FAKE, None) == -1
        assert fn(ok, 0, FAKE, FAKE, ODD, None) == -1
        assert fn(z, 0, None, None, None, None) == 0
    assert lib.moe_unpermute(ok, 0, None, FAKE, FAKE, FAKE, None) == -1
    assert lib.moe_unpermute(ok, 0, FAKE, FAKE, None, FAKE, None) == -1
    assert lib.moe_unpermute(ok, 0, FAKE, FAKE, FAKE, ODD, None) == -1
    assert lib.moe_unpermute(z, 0, None, None, None, None, None) == 0
    ub = lib.moe_unpermute_backward
    assert ub(ok, 0, None, FAKE, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert ub(ok, 0, FAKE, None, FAKE, FAKE, FAKE, FAKE, None) == -1   # dtopk_w needs rows
    assert ub(ok, 0, FAKE, FAKE, FAKE, None, FAKE, FAKE, None) == -1
    assert ub(ok, 0, FAKE, FAKE, FAKE, FAKE, None, None, None) == -1   # nothing to write
    assert ub(ok, 0, FAKE, FAKE, FAKE, FAKE, ODD, FAKE, None) == -1
    assert ub(ok, 3, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert ub(z, 0, None, None, None, None, None, None, None) == 0


def test_adapter_shapes(lib):
    assert moe.moe_adapter_check(moe.AdapterShape(**AD)) == 0
    bad = [({"T": -1}, -1), ({"H": 0}, -1), ({"N": 0}, -1), ({"L": 0}, -1), ({"rank": 0}, -1),
           ({"H": 192}, -2), ({"H": (1 << 17) + 128}, -2), ({"N": 12}, -2),
           ({"N": (1 << 20) + 8}, -2), ({"rank": 12}, -2), ({"rank": 264}, -2),
           ({"L": (1 << 24) + 1}, -2),
           ({"T": 1 << 23, "H": 512}, -2), ({"T": 1 << 23, "H": 128, "N": 512}, -2)]
    for kw, code in bad:
        s = moe.AdapterShape(**{**AD, **kw})
        assert moe.moe_adapter_check(s) == code, kw
        assert moe.moe_adapter_workspace_size(s) == 0
        assert lib.moe_adapter_project(ctypes.byref(s.c()), 0, *([FAKE] * 9), 1 << 40,
                                       None) == code
    assert lib.moe_adapter_check(None) == -1
    assert moe.moe_adapter_workspace_size(moe.AdapterShape(**{**AD, "T": 0})) == 0
    assert moe.moe_adapter_workspace_size(moe.AdapterShape(**AD)) >= 16 * 16 * 4


def test_adapter_refusals(lib):
    f, ok = lib.moe_adapter_project, a_shape()

    def args(**kw):
        v = dict(x=FAKE, w=FAKE, base=None, ids=FAKE, a=FAKE, b=FAKE, scale=FAKE, out=FAKE,
                 ws=FAKE, n=1 << 30)
        v.update(kw)
        return [*v.values(), None]

    assert f(ok, 2, *args()) == -1                        # float32 rows
    for name in ("x", "ids", "a", "b", "out"):
        assert f(ok, 0, *args(**{name: None})) == -1, name
    for name in ("x", "w", "a", "b", "out"):
        assert f(ok, 0, *args(**{name: ODD})) == -1, name
    assert f(ok, 0, *args(base=FAKE)) == -1               # both
    assert f(ok, 0, *args(w=None)) == -1                  # neither
    assert f(ok, 0, *args(w=None, base=ODD)) == -1
    assert f(ok, 0, *args(ws=None)) == -3
    assert f(ok, 0, *args(n=16)) == -3
    assert f(ok, 0, *args(ws=ctypes.c_void_p(256 + 16))) == -3
    assert f(a_shape(T=0), 0, *args(x=None, w=None, ids=None, ws=None)) == 0
    assert "adapters" in moe.moe_strerror(-2)


def test_binding_refuses_tensors(lib):
    """Wrong type, wrong shape, not contiguous, not on a GPU: refused in Python."""
    s = moe.MoeShape(T=4, H=128, I=128, K=2, E_total=8, E_local=8)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    rr = torch.zeros(8, dtype=torch.int32)
    rows = torch.zeros(8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_permute(s, x, rr, rows)                   # host tensors
    with pytest.raises(TypeError):
        moe.moe_permute(s, x.double(), rr, rows)
    with pytest.raises(TypeError):
        moe.moe_permute(s, None, rr, rows)
    with pytest.raises(ValueError):
        moe.moe_unpermute_backward(s, x, rows, None, rr, None, None)
    with pytest.raises(ValueError):
        moe.moe_route(s, torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32),
                      torch.zeros(4, 2))
    a = moe.AdapterShape(T=4, H=128, N=8, L=1, rank=8)
    with pytest.raises(TypeError):
        moe.moe_adapter_project(a, x.float(), None, rr, rows, rows, None, x, rr)
    with pytest.raises(ValueError):
        moe.moe_adapter_project(a, x, None, rr, rows, rows, None, x, rr)


def test_shapes_copy_after_use(lib):
    """What a shape object keeps for its calls does not stand in the way of copies."""
    import copy
    import pickle
    s = moe.AdapterShape(**AD)
    assert moe.moe_adapter_check(s) == 0
    m = moe.MoeShape(**V4)
    assert moe._row_sizes(m)[1] == (128 * 6, 7168) and moe._ref(m) is moe._ref(m)
    for v in (s, m):
        for w in (copy.deepcopy(v), pickle.loads(pickle.dumps(v))):
            assert w == v and hash(w) == hash(v)


def test_shapes_keep_only_their_sizes_in_sight(lib):
    """vars() of a shape that calls have used makes a shape again, and asdict() and replace()
    do."""
    import dataclasses
    for v, n in ((moe.MoeShape(**V4), "T"), (moe.AdapterShape(**AD), "T")):
        moe._ref(v)
        if isinstance(v, moe.MoeShape):
            moe._row_sizes(v)
        assert type(v)(**vars(v)) == v and type(v)(**dataclasses.asdict(v)) == v
        other = dataclasses.replace(v, T=v.T + 1)
        assert moe._ref(other) is not moe._ref(v) and moe._ref(v) is moe._ref(v)
        assert moe._ref(other)._obj.T == v.T + 1
