"""What makes the binding's native part stale, without a GPU."""
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def build():
    from dequantisation_fp8q_token_b200 import build as b
    b.build()
    return b


def test_the_torch_extension_is_current_after_a_build(build):
    assert build.torch_ext_up_to_date()
    from dequantisation_fp8q_token_b200 import ffn
    assert ffn._native().built_for == build.torch_ext_tag()


@pytest.mark.parametrize("what", ["torch", "abi", "python"])
def test_it_is_stale_under_another_torch_or_python(build, monkeypatch, what):
    """A module built against another torch, another C++ ABI or another Python is built again, although its
    sources are older than it is."""
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif what == "abi":
        abi = torch.compiled_with_cxx11_abi()
        monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: not abi)
    else:
        monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-30")
    assert not build.torch_ext_up_to_date()
    monkeypatch.undo()
    assert build.torch_ext_up_to_date()
