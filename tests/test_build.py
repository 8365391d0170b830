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


def test_library_is_built_where_the_binding_cannot_be(monkeypatch, tmp_path, capsys):
    """The C library does without the headers of Python and torch; what the binding lacks is named where the binding is
    asked for."""
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "binding.so"))
    lib = build.build()
    assert lib == build.LIB and os.path.exists(lib)
    with pytest.raises(RuntimeError, match="no-such-compiler"):
        build.build_binding()
    assert build.main([]) == 0
    out = capsys.readouterr()
    assert build.LIB in out.out and "the Python binding was not built" in out.err
    assert os.listdir(tmp_path) == []
