"""The library is built with or without torch and whatever comes of its Python
binding, which is built again for another torch.  The compilers are stand-ins
that write their output's name into it."""
import os
import stat

import pytest

from dynamic_sparsity_spmspv_gb300 import _build

TOOL = """#!/bin/sh
for a in "$@"; do
    case "$a" in *binding.cpp) {binding} ;; esac
    [ "$prev" = -o ] && out="$a"
    prev="$a"
done
echo "$out" > "$out"
echo "$out" >> {log}
"""


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """A build folder of its own and stand-ins for nvcc and g++; returns a function that sets what compiling the binding
    does, and the list of what was made."""
    bin_, out, log = tmp_path / "bin", tmp_path / "out", tmp_path / "log"
    bin_.mkdir()

    def binding(does=":"):
        for name in ("nvcc", "g++"):
            p = bin_ / name
            p.write_text(TOOL.format(binding=does, log=log))
            p.chmod(p.stat().st_mode | stat.S_IXUSR)

    def made():
        names = [os.path.basename(l).split(".tmp")[0] for l in log.read_text().split()] if log.exists() else []
        log.write_text("")
        return names

    binding()
    monkeypatch.setenv("PATH", f"{bin_}:{os.environ['PATH']}")
    monkeypatch.setattr(_build, "NVCC", str(bin_ / "nvcc"))
    monkeypatch.setattr(_build, "OUT", str(out))
    monkeypatch.setattr(_build, "LIB", str(out / "libdbspmspv.so"))
    monkeypatch.setattr(_build, "OPS", str(out / "_dbsops.so"))
    return binding, made


def test_both_are_built_and_then_left(tools):
    _, made = tools
    _build.build()
    names = made()
    assert os.path.exists(_build.LIB) and os.path.exists(_build.OPS) and "binding.cpp.o" in names and "attention.cu.o" in names
    _build.build()
    assert made() == []


def test_the_library_needs_no_torch(tools, monkeypatch):
    import importlib.util
    _, made = tools
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    _build.build()
    names = made()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.OPS) and "binding.cpp.o" not in names
    _build.build()
    assert made() == []


def test_the_library_is_there_where_the_binding_fails(tools):
    binding, made = tools
    binding("echo no such header; exit 1")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.OPS)
    made()
    binding()
    _build.build()
    assert os.path.exists(_build.OPS) and "attention.cu.o" not in made()


def test_another_torch_gets_another_binding(tools, monkeypatch):
    import importlib.metadata
    _, made = tools
    _build.build()
    made()
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0")
    _build.build()
    names = made()
    assert "binding.cpp.o" in names and "_dbsops.so" in names and "attention.cu.o" not in names
    _build.build()
    assert made() == []
