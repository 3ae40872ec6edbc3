"""What gets built, and when, without compiling anything."""
import importlib.metadata
import importlib.util
import os

import pytest

from exact_io_aware_100_b200 import build


@pytest.fixture
def ran(tmp_path, monkeypatch):
    """The commands that a build in an empty place runs; each writes its target."""
    commands = []

    def run(cmd, **_):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return type("Done", (), {"returncode": 0, "stdout": "", "stderr": ""})

    for name in ("LIB", "EXT", "EXT_FOR"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    monkeypatch.setattr(build.subprocess, "run", run)
    return commands


def test_the_c_library_needs_no_torch(ran, monkeypatch, capsys):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert not build.up_to_date()
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert len(ran) == 1 and not any("torch" in x for x in ran[0])
    assert "_serving.so" in capsys.readouterr().err and not os.path.exists(build.EXT)
    assert build.up_to_date()
    build.build()
    assert len(ran) == 1


def test_a_torch_without_cuda_is_none(ran, tmp_path, monkeypatch):
    spec = type("Spec", (), {"submodule_search_locations": [str(tmp_path)]})
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec)
    build.build()
    assert len(ran) == 1


def test_the_binding_is_rebuilt_for_another_torch_or_python(ran, monkeypatch):
    build.build()
    assert [c[c.index("-o") + 1] for c in ran] == [build.LIB, build.EXT] and build.up_to_date()
    build.build()
    assert len(ran) == 2                                                       # nothing to do
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0")
    assert not build.up_to_date()
    build.build()
    assert len(ran) == 3 and ran[2][ran[2].index("-o") + 1] == build.EXT and build.up_to_date()


def test_nothing_is_looked_for_when_all_is_built(ran, monkeypatch):
    build.build()
    monkeypatch.setattr(build, "nvcc_path", lambda: pytest.fail("no compiler is needed"))
    build.build()
    assert len(ran) == 2


def test_a_binding_that_does_not_load_is_named(monkeypatch):
    import sys

    from exact_io_aware_100_b200 import serving
    monkeypatch.setattr(serving, "_ext", None)
    monkeypatch.setitem(sys.modules, "exact_io_aware_100_b200._serving", None)     # its import fails
    monkeypatch.delattr(sys.modules["exact_io_aware_100_b200"], "_serving", raising=False)
    build.build()
    with pytest.raises(RuntimeError, match="does not load with this Python and torch"):
        serving._native()
    monkeypatch.setattr(build, "EXT", "/nowhere/_serving.so")
    with pytest.raises(RuntimeError, match="is not built"):
        serving._native()
