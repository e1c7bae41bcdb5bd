"""The compiled binding of the paged cache's calls is optional: the library is built without it."""
import importlib.util
import os
import sysconfig

import pytest

from long_context_indexing_b200 import _build


@pytest.fixture
def places(tmp_path, monkeypatch):
    """Builds into a folder of their own, with an old binding in it (objects are the tree's)."""
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "liblsa.so"))
    name = os.path.basename(_build.BINDING)
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / name))
    for n in {name, "_paged_binding.so"}:
        (tmp_path / n).write_bytes(b"old")
        os.utime(tmp_path / n, (0, 0))
    return tmp_path


def _assert_library_alone(places, capsys):
    assert _build.build() == str(places / "liblsa.so")
    assert os.listdir(places) == ["liblsa.so"]           # no old binding is left to be loaded
    assert "no compiled binding" in capsys.readouterr().err


def test_library_is_built_where_the_compiler_fails(places, monkeypatch, capsys):
    monkeypatch.setattr(_build, "CXX", "false")
    _assert_library_alone(places, capsys)


def test_library_is_built_without_a_compiler(places, monkeypatch, capsys):
    monkeypatch.setattr(_build, "CXX", str(places / "nowhere"))
    _assert_library_alone(places, capsys)


def test_library_is_built_without_torch(places, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    _assert_library_alone(places, capsys)


def test_binding_is_of_this_python_alone(places):
    assert _build.BINDING.endswith("_paged_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
    _build.build()
    assert sorted(os.listdir(places)) == sorted(["liblsa.so", os.path.basename(_build.BINDING)])
