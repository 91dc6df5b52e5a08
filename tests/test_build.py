"""The build's steps, with stand-ins for the compilers: the library needs neither torch nor the host
compiler."""
import os
import stat
import sys

import pytest


@pytest.fixture
def kbuild(tmp_path, monkeypatch):
    from gated_delta_rule_59_amd import build

    def compiler(name, fails=False):
        """Writes what it is asked for with -o, or fails."""
        path = tmp_path / name
        path.write_text("#!/bin/sh\n" + ("echo no such header; exit 1\n" if fails else
                        'while [ "$1" != -o ]; do shift; done; echo built > "$2"\n'))
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        return str(path)

    build.compiler = compiler
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "HIPCC", compiler("hipcc"))
    monkeypatch.setattr(build, "CXX", compiler("cxx"))
    yield build
    del build.compiler


def test_both_modules(kbuild):
    assert kbuild.build() == kbuild.LIB
    assert os.path.exists(kbuild.LIB) and os.path.exists(kbuild.MARSHAL)


def test_without_torch(kbuild, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    kbuild.build()
    assert os.path.exists(kbuild.LIB) and not os.path.exists(kbuild.MARSHAL)
    assert "_marshal.so is not built" in capsys.readouterr().err


def test_a_host_compiler_that_fails(kbuild, monkeypatch):
    monkeypatch.setattr(kbuild, "CXX", kbuild.compiler("bad", fails=True))
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        kbuild.build()
    assert os.path.exists(kbuild.LIB) and not os.path.exists(kbuild.MARSHAL)


def test_a_device_compiler_that_fails(kbuild, monkeypatch):
    monkeypatch.setattr(kbuild, "HIPCC", kbuild.compiler("bad", fails=True))
    with pytest.raises(RuntimeError, match="compiler failed"):
        kbuild.build()
    assert not os.path.exists(kbuild.LIB)
