"""What the feed-forward block and the residual joint accept, without a GPU's work: calls of no
rows, one workspace for many sizes, and the largest sizes there are."""

import pytest

import dispatch_grouped_gemm_amd as moe
from dispatch_grouped_gemm_amd import _build
from test_ffn_refusals import FAKE, FF, NO, f_shape, n_shape


@pytest.fixture(scope="module")
def lib():
    _build.build(force=False)
    return moe.lib()


def test_no_rows_and_frozen_weights(lib):
    """The gradients of no rows, none of the weights' asked for: an empty tensor's pointer is
    NULL, and that is not a call without outputs."""
    none = [None] * 16
    assert lib.moe_ffn_backward(f_shape(T=0), 0, *none[:10], 0, 0, None, 0, None) == 0
    # ... with the weights at hand and kept rows in 8 bits
    assert lib.moe_ffn_backward(f_shape(T=0), 0, None, None, None, FAKE, FAKE, None, None, None,
                                None, None, 0, 1, FAKE, 1 << 20, None) == 0
    assert lib.moe_norm_backward(n_shape(T=0), 0, *none[:13], 0, None) == 0
    assert lib.moe_norm_backward(n_shape(T=0), 0, None, None, None, None, FAKE, None, FAKE,
                                 *none[:6], 0, None) == 0
    # of some rows it is one
    assert lib.moe_ffn_backward(f_shape(), 0, *([FAKE] * 7), None, None, None, 0, 0, FAKE,
                                1 << 30, None) == -1
    assert lib.moe_norm_backward(n_shape(), 0, *([FAKE] * 7), *none[:5], FAKE, 1 << 30,
                                 None) == -1


@pytest.mark.parametrize("H,I", [(5120, 2304), (2304, 1408), (7168, 18432), (7168, 2048),
                                 (96, 64), (2304, 96), (1632, 352), (32, 32), (64, 131072)])
def test_a_workspace_serves_fewer_rows(lib, H, I):
    """Parts of K come and go with the rows; the workspace of many rows has room for all of
    them (a server keeps the one of its largest batch)."""
    rows = sorted({*range(1, 700), *range(700, 3000, 31), 4096, 8191, 65536, 1 << 20})
    for backward in (False, True):
        before = 0
        for T in rows:
            n = moe.moe_ffn_workspace_size(moe.FfnShape(T=T, H=H, I=I), backward)
            assert n >= before, (T, backward)
            before = n


def test_the_largest_sizes(lib):
    for kw, code in [(dict(T=1 << 21), 0), (dict(T=(1 << 21) + 1), -2), (dict(H=1 << 14), 0),
                     (dict(H=(1 << 14) + 32), -2)]:
        assert moe.moe_norm_check(moe.NormShape(**{**NO, **kw})) == code, kw
    for kw, code in [(dict(T=1 << 24), 0), (dict(T=(1 << 24) + 1), -2), (dict(H=1 << 17), 0),
                     (dict(H=(1 << 17) + 32), -2), (dict(I=1 << 17), 0),
                     (dict(I=(1 << 17) + 32), -2)]:
        assert moe.moe_ffn_check(moe.FfnShape(**{**FF, **kw})) == code, kw
