"""The tensor types that the binding takes, with a torch that lacks one."""
import pytest
import torch

from test_abi import lib  # noqa: F401  (the module's build-and-load fixture)
from test_binding import fresh  # noqa: F401


@pytest.fixture
def without_e8m0(fresh, monkeypatch):  # noqa: F811
    monkeypatch.delattr(torch, "float8_e8m0fnu", raising=False)
    monkeypatch.setattr(fresh, "_E8M0", set())
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    return fresh


def test_a_torch_without_e8m0(without_e8m0):
    """The calls that existed before block scales, and scales as uint8 codes, need no torch.float8_e8m0fnu."""
    lib = without_e8m0  # noqa: F811
    lib._load_torch()
    assert lib._torch is torch and lib._E8M0 == {torch.uint8}
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(lib.QffnError) as e:                         # (refused for its device, not for its type)
        lib.qffn_linear(x, None, x, x, None, None, 0, 4, 64, 64, None, stream=0)
    assert e.value.status == 1
