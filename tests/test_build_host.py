"""What the build makes and survives, with stand-ins for the compilers."""
import os
import subprocess

import pytest

from linear_attention_recurrence_02_gb300 import build


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """nvcc writes what it is asked for; the C compiler answers as `compilers.c` says. Outputs go to tmp_path."""
    class State:
        c, commands = 0, []

    def run(cmd, **_):
        State.commands.append(cmd)
        code = 0 if cmd[0] == "/nvcc" else State.c
        if code == 0:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("x")
        return subprocess.CompletedProcess(cmd, code, "", "" if code == 0 else "fatal error: Python.h: No such file")

    State.commands = []
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / os.path.basename(build.FASTCALL)))
    monkeypatch.setattr(build, "_nvcc", lambda: "/nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setenv("CC", "gcc")
    return State


def test_the_library_does_not_need_the_extension(compilers, monkeypatch):
    """No Python.h, then no C compiler at all: libkda.so is linked and a warning names what is missing; the
    next build tries the extension again and leaves the library alone."""
    compilers.c = 1
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build_library() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.FASTCALL) and not build.up_to_date()
    monkeypatch.delenv("CC")
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    compilers.commands.clear()
    with pytest.warns(UserWarning, match="no C compiler"):
        build.build_library()
    assert compilers.commands == []
    compilers.c = 0
    monkeypatch.setenv("CC", "gcc")
    build.build_library()
    assert len(compilers.commands) == 1 and os.path.exists(build.FASTCALL) and build.up_to_date()
    compilers.commands.clear()
    build.build_library()
    assert compilers.commands == []


def test_a_library_that_does_not_compile_is_an_error(compilers, monkeypatch):
    monkeypatch.setattr(build.subprocess, "run",
                        lambda cmd, **_: subprocess.CompletedProcess(cmd, 1, "", "error: no"))
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build_library()


def test_the_c_compiler_may_come_with_arguments(compilers, monkeypatch):
    monkeypatch.setenv("CC", "ccache gcc -pthread")
    build.build_library()
    assert [c[:3] for c in compilers.commands if c[0] != "/nvcc"] == [["ccache", "gcc", "-pthread"]]


def test_the_extension_belongs_to_one_interpreter():
    """Its name ends in this interpreter's suffix, so that another Python builds its own instead of loading it."""
    import sysconfig
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert "cpython" in suffix and os.path.basename(build.FASTCALL) == "kda_fastcall" + suffix
