"""Building in-tree: what is compiled, where it goes and when a built file is taken (no GPU)."""
import os

import pytest
import torch

import prefill_sigmoid_top_b200 as moe
from prefill_sigmoid_top_b200 import build


def test_binding_of_another_torch_is_not_loaded(monkeypatch):
    """The binding is compiled against torch's C++ headers: after a change of version the one on disk is built anew."""
    moe._load_binding()
    assert moe._fast.__file__ == build.binding_path() and os.path.exists(build.binding_path())

    class Built(Exception):
        pass

    def builder(force=False):
        raise Built

    monkeypatch.setattr(moe, "_fast", None)
    monkeypatch.setattr(build, "build_binding", builder)
    moe._load_binding()  # the same version: as it stands
    monkeypatch.setattr(moe, "_fast", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    with pytest.raises(Built):
        moe._load_binding()
