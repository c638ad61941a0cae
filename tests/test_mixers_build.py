"""The mixers' binding as a built file: which library it loads, when it is built again.  No GPU."""
import importlib.metadata
import os
import shutil
import subprocess
import sys

import pytest

from chunk_gated_delta_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_a_copied_tree_loads_its_own_library(tmp_path):
    """The package copied elsewhere: its binding uses the library that lies beside it, the one that the
    package's other calls use, so that their status words are the same ones."""
    pkg = tmp_path / "chunk_gated_delta_b200"
    pkg.mkdir()
    for f in os.listdir(build.PKG):
        if f.endswith((".py", ".so")):
            shutil.copy(os.path.join(build.PKG, f), pkg / f)
    code = ("from chunk_gated_delta_b200 import mixers, load, library_path\n"
            "load(); mixers._bind()\n"
            "print(*sorted({l.split()[-1] for l in open('/proc/self/maps') if 'libcarve.so' in l}))\n")
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    got = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env, capture_output=True, text=True, check=True).stdout.split()
    assert got == [str(pkg / "libcarve.so")]


def test_a_binding_of_another_pytorch_or_python_is_built_again(monkeypatch):
    assert not build.bind_stale()
    calls = []
    monkeypatch.setattr(build, "_bind", lambda verbose: calls.append(1))
    for other in ("torch 0.1 .so", build.bind_for() + "x", ""):
        monkeypatch.setattr(build, "bind_for", lambda other=other: other)
        assert build.bind_stale()
        assert build.build() == build.LIB and calls.pop() and not calls


def test_without_pytorch_the_library_is_built_alone(monkeypatch):
    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(importlib.metadata, "version", missing)
    monkeypatch.setattr(build, "BIND", build.BIND + ".none")
    monkeypatch.setattr(build, "_compile", lambda src, *a: build._obj(src))
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, check: open(cmd[cmd.index("-o") + 1], "w").close())
    monkeypatch.setattr(build, "LIB", build.LIB + ".none")
    try:
        assert not build.bind_stale()
        for force in (False, True):
            assert build.build(force=force) == build.LIB
            assert not os.path.exists(build.BIND)
    finally:
        if os.path.exists(build.LIB):
            os.unlink(build.LIB)
