"""The build's steps, with the compilers replaced: what is built where torch is missing."""
import importlib.util
import os
import shutil

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mass_gated_causal_b200")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources without anything built, and the build module over it with its commands recorded."""
    shutil.copytree(os.path.join(PACKAGE, "csrc"), tmp_path / "p" / "csrc")
    shutil.copytree(os.path.join(os.path.dirname(PACKAGE), "include"), tmp_path / "include")
    shutil.copy(os.path.join(PACKAGE, "build.py"), tmp_path / "p" / "build.py")
    spec = importlib.util.spec_from_file_location("copied_build", str(tmp_path / "p" / "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build.subprocess, "check_call", run)
    return build, commands


def test_the_c_library_is_built_without_torch(tree, monkeypatch, capsys):
    build, commands = tree
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))
    monkeypatch.setitem(__import__("sys").modules, "torch", None)  # an import of it fails
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_LIB)
    assert len(commands) == len(build.sources()) + 1 and not any("g++" in c[0] for c in commands)
    assert "mala_torch.so" in capsys.readouterr().out
    assert not build.needs_build()  # and not again


def test_both_are_built_with_torch(tree):
    build, commands = tree
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.TORCH_LIB)
    assert len(commands) == len(build.sources()) + 2
    assert not build.needs_build()
    build.build()
    assert len(commands) == len(build.sources()) + 2
    later = os.path.getmtime(build.LIB) + 10
    os.utime(os.path.join(build.SRC_DIR, "mala_rope.cuh"), (later, later))  # one unit's header
    assert build.needs_build()
    build.build()
    assert len(commands) == len(build.sources()) + 2 + 2  # that unit and the link
