"""A binding that does not compile (another torch, no g++) costs the calls that need it, not the
library."""
import os
import stat

import pytest

from paged_kv_cache_70_gb300 import build as B


@pytest.fixture
def folder(tmp_path, monkeypatch):
    """Builds into a folder of its own, with an nvcc that only makes its outputs."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\ntouch "$2"\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    out = tmp_path / "out"
    monkeypatch.setattr(B, "_nvcc", lambda: str(nvcc))
    monkeypatch.setattr(B, "BUILD", str(out))
    monkeypatch.setattr(B, "LIB", str(out / "libpagedkv.so"))
    return tmp_path


def broken_compiler(folder, monkeypatch):
    cxx = folder / "bin" / "g++"
    cxx.parent.mkdir()
    cxx.write_text('#!/bin/sh\necho "no such header" >&2\nexit 1\n')
    cxx.chmod(cxx.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("PATH", f"{cxx.parent}{os.pathsep}{os.environ['PATH']}")


def test_the_library_is_built_without_the_binding(folder, monkeypatch, capsys):
    broken_compiler(folder, monkeypatch)
    lib = B.build()
    assert os.path.exists(lib)
    assert not os.path.exists(B.binding_path())
    err = capsys.readouterr().err
    assert "no such header" in err and all(name in err for name in B.BINDING_CALLS)


def test_a_binding_of_an_older_source_is_not_left(folder, monkeypatch):
    broken_compiler(folder, monkeypatch)
    os.makedirs(B.BUILD)
    with open(B.binding_path(), "w"):
        pass
    os.utime(B.binding_path(), (0, 0))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        B.build_binding()
    assert not os.path.exists(B.binding_path())
