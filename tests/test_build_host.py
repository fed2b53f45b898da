"""The build without what only the serving operators' binding needs."""
import os

import pytest

from test_activation_aware_amd import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one host source, in a folder of its own; a binding of an earlier build beside it."""
    (tmp_path / "one.cpp").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "sources", lambda: [str(tmp_path / "one.cpp")])
    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    (tmp_path / "_binding.so").write_text("of an earlier build")
    return build


def missing_compiler():
    raise FileNotFoundError("g++")


@pytest.mark.parametrize("binding", [missing_compiler, lambda: (build.BINDING, 1, "g++ ...", "no such header")])
def test_the_library_is_built_without_the_binding(small, monkeypatch, binding):
    monkeypatch.setattr(small, "_compile_binding", binding)
    with pytest.warns(RuntimeWarning, match="_binding.so.*(g\\+\\+|no such header)"):
        assert small.build() == small.LIB
    assert os.path.getsize(small.LIB) > 0
    assert not os.path.exists(small.BINDING)  # the earlier one may not fit this library


def test_a_library_that_does_not_compile_is_an_error(small, monkeypatch, tmp_path):
    monkeypatch.setattr(small, "_compile_binding", lambda: (build.BINDING, 0, "", ""))
    (tmp_path / "one.cpp").write_text("not C++\n")
    with pytest.raises(RuntimeError, match="compiler failed"):
        small.build()
