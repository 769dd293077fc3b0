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
