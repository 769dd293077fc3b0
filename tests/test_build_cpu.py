"""Building the library where its argument filler cannot be built."""
import importlib.util
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """A fresh copy of the build module, the filler's target somewhere else; the library itself is built."""
    sys.path.insert(0, ROOT)
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("_hm_build_test",
                                                  os.path.join(ROOT, "selective_ssm_sequence_b200", "_build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "MARSHAL", str(tmp_path / "_marshal.so"))
    return mod


def test_the_library_stands_without_its_filler(builder, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.warns(RuntimeWarning, match="_marshal.so was not built"):
        assert builder.build() == builder.LIB
    assert not os.path.exists(builder.MARSHAL)


def test_the_library_comes_first(builder, monkeypatch):
    """It is there even where the filler's build does not return."""
    at = []
    monkeypatch.setattr(builder, "build_marshal", lambda force: at.append(os.path.exists(builder.LIB)))
    monkeypatch.setattr(builder, "_stale", lambda target, deps: at.append(target) and False)
    builder.build()
    assert at[-1] is True and builder.LIB in at[:-1]


def test_the_filler_is_rebuilt_for_another_torch(builder, tmp_path, monkeypatch):
    """Built once it is fresh; with another torch, or a stamp that is not there, it is not."""
    monkeypatch.setattr(builder, "OBJDIR", str(tmp_path))
    builder.build_marshal()
    at = os.path.getmtime(builder.MARSHAL)
    monkeypatch.setenv("CXX", "/bin/false")
    assert builder.build_marshal() == builder.MARSHAL and os.path.getmtime(builder.MARSHAL) == at
    monkeypatch.setattr(builder, "marshal_tag", lambda: "torch 0 abi 0 cpython-0")
    with pytest.raises(RuntimeError, match="/bin/false"):
        builder.build_marshal()


def test_a_filler_of_another_torch_is_not_used(builder, monkeypatch):
    import torch
    import selective_ssm_sequence_b200 as hm
    monkeypatch.setattr(hm, "_native", None)
    assert hm._filler().built_for.startswith("torch " + torch.__version__)
    monkeypatch.setattr(hm, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.0")
    with pytest.warns(RuntimeWarning, match="another torch"):
        assert hm._filler().gated_step() is None
