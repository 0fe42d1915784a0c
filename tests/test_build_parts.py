"""build_lib.build() with stand-in compilers (shell scripts that write their
output file): the library does not depend on what the binding's native part
needs, and a native part of an older build does not outlive the library."""
import os
import shutil
import stat

import pytest

from w4a4_quantized_linear_cube_amd import build_lib

TOOL = """#!/bin/sh
case " $* " in *{fails}*) echo no such thing; exit 1;; esac
while [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done
"""


def _tool(path, fails="a-word-that-no-command-has"):
    path.write_text(TOOL.format(fails=fails))
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    tools = tmp_path / "tools"
    tools.mkdir()
    for name in ("sh", "echo"):
        os.symlink(shutil.which(name), tools / name)
    monkeypatch.setenv("PATH", str(tools))
    monkeypatch.setattr(build_lib, "HIPCC", _tool(tools / "hipcc"))
    for name, path in (("BUILD", "_build"), ("LIB", "libdq.so"), ("CALL_LIB", "_dqcall.so")):
        monkeypatch.setattr(build_lib, name, str(tmp_path / path))
    (tmp_path / "_dqcall.so").write_text("older\n")
    return tmp_path


def test_both_parts(tree):
    _tool(tree / "tools" / "g++")
    assert build_lib.build() == str(tree / "libdq.so")
    assert (tree / "libdq.so").read_text() == (tree / "_dqcall.so").read_text() == "built\n"


def test_without_a_host_compiler(tree, capsys):
    assert build_lib.build() == str(tree / "libdq.so")
    assert (tree / "libdq.so").read_text() == "built\n" and not (tree / "_dqcall.so").exists()
    assert "g++" in capsys.readouterr().err


def test_without_torch(tree, monkeypatch, capsys):
    import importlib.util
    _tool(tree / "tools" / "g++")
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    assert build_lib.build() == str(tree / "libdq.so")
    assert (tree / "libdq.so").read_text() == "built\n" and not (tree / "_dqcall.so").exists()
    assert "torch" in capsys.readouterr().err


@pytest.mark.parametrize("fails", ["binding.cpp", "-shared"])
def test_an_error_in_the_native_part_is_one(tree, fails):
    """... but the library is there by then."""
    _tool(tree / "tools" / "g++", fails)
    with pytest.raises(RuntimeError, match="_dqcall"):
        build_lib.build()
    assert (tree / "libdq.so").read_text() == "built\n" and not (tree / "_dqcall.so").exists()


def test_an_error_in_the_library_is_one(tree, monkeypatch):
    _tool(tree / "tools" / "g++")
    monkeypatch.setattr(build_lib, "HIPCC", _tool(tree / "tools" / "hipcc", "norm.hip"))
    with pytest.raises(RuntimeError, match="norm.hip"):
        build_lib.build()
    assert not (tree / "libdq.so").exists()
