"""build.py with stand-ins for the compilers: what is installed when a part of the build is missing or fails."""
import importlib.util
import os
import stat

import pytest

from convolution_implicit_gemm_fwd_amd import build

GOOD = '#!/bin/sh\nwhile [ $# -gt 1 ]; do [ "$1" = -o ] && echo made > "$2"; shift; done\n'
BAD = "#!/bin/sh\necho no such header\nexit 1\n"


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Stand-ins `hipcc` and `cxx` that succeed, and an empty folder for what is built."""
    out = tmp_path / "package"
    out.mkdir()
    for name in ("hipcc", "cxx"):
        write(tmp_path / name, GOOD)
    monkeypatch.setenv("HIPCC", str(tmp_path / "hipcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "cxx"))
    for name, value in dict(PKG=out, LIB=out / "libconvimg.so", EXT=out / "_rows.so").items():
        monkeypatch.setattr(build, name, str(value))
    return tmp_path


def write(path, text):
    path.write_text(text)
    os.chmod(path, stat.S_IRWXU)


def built(tree):
    return sorted(os.listdir(tree / "package"))


def without(monkeypatch, module):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == module else find(name, *a))


def test_both_are_installed(tree):
    assert build.build() == build.LIB
    assert built(tree) == ["_rows.so", "libconvimg.so"]


def test_the_library_needs_no_torch(tree, monkeypatch):
    without(monkeypatch, "torch")
    assert build.build() == build.LIB
    assert built(tree) == ["libconvimg.so"]


def test_a_failing_torch_module_leaves_the_library(tree):
    write(tree / "cxx", BAD)
    with pytest.raises(RuntimeError, match="_rows.so(.|\n)*no such header"):
        build.build()
    assert built(tree) == ["libconvimg.so"]


def test_a_failing_library_installs_nothing(tree):
    write(tree / "hipcc", BAD)
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert built(tree) == []


def test_a_missing_compiler_of_the_torch_module_leaves_the_library(tree, monkeypatch):
    monkeypatch.setenv("CXX", str(tree / "none"))
    with pytest.raises(RuntimeError):
        build.build()
    assert built(tree) == ["libconvimg.so"]
