"""The binding's comparisons of one tensor: the built ones are loaded only for the torch and the
Python that they were built for, and the plain ones that take their place say the same."""

import shutil

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
from dispatch_grouped_gemm_amd import _build


@pytest.fixture
def built():
    _build.build(force=False)


def test_built_for_this_torch(built):
    assert _build.checks_current() and not _build._stale()


@pytest.mark.parametrize("version", ["0.1", torch.__version__ + "0", torch.__version__[:-1]])
def test_another_torch(built, monkeypatch, version):
    monkeypatch.setattr(torch, "__version__", version)
    assert not _build.checks_current() and _build._stale()
    monkeypatch.setattr(moe, "_address", moe._address_first)
    with pytest.warns(UserWarning, match="another torch"):
        assert moe._address(torch.zeros(4), (4,), torch.float32, 0) == -1
    assert moe._address is moe._address_plain


def test_the_library_alone(built, monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "CHECKS", str(tmp_path / "_checks.so"))
    monkeypatch.setattr(moe, "_address", moe._address_first)
    assert moe._address(None, (4,), torch.float32, 0) == -1
    assert moe._address is moe._address_plain
    with pytest.raises(ValueError):
        moe.moe_norm_forward(moe.NormShape(T=4, H=64), torch.zeros(4, 64), torch.zeros(64),
                             torch.zeros(4, 64))
    # a copy of the built ones is found to be
    shutil.copy(_build.os.path.join(_build.HERE, "_checks.so"), tmp_path / "_checks.so")
    assert _build.checks_current()


@pytest.mark.gpu
def test_plain_and_built_alike():
    from dispatch_grouped_gemm_amd._checks import address
    bf, dev = torch.bfloat16, "cuda"
    t = torch.zeros(6, 64, dtype=bf, device=dev)
    for v, as_wanted in ((t, True), (t[:6], True), (t[1:5], False), (t.float(), False),
                         (t[:, :32], False), (t.t(), False), (t.cpu(), False), (None, False),
                         (t.reshape(-1), False), (t.reshape(6, 8, 8), False), (3, False),
                         (torch.zeros(64, 6, dtype=bf, device=dev).t(), False),
                         (torch.nn.Parameter(t), True), (t.to_sparse(), False),
                         (t.as_strided((6, 64), (0, 1)), False)):
        a, b = [f(v, (6, 64), bf, t.device.index) for f in (address, moe._address_plain)]
        assert a == b and (a >= 0) == as_wanted
        assert not as_wanted or a == v.data_ptr()
        assert address(v, (6, 64), bf, 1) == moe._address_plain(v, (6, 64), bf, 1) == -1
    e = torch.empty(0, 64, dtype=bf, device=dev)
    assert address(e, (0, 64), bf, 0) == moe._address_plain(e, (0, 64), bf, 0) == 0
