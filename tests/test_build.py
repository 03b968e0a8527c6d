"""What build() makes and when it makes it again, with stand-ins for the compilers
(and, for the built files, the real ones; no GPU needed)."""
import os
import shutil
import subprocess
import sys
import sysconfig
from types import SimpleNamespace

import pytest

from bit_quantized_expert_moe_gb300 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build() with its outputs under tmp_path and compilers that make empty files;
    returns the commands that were run."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        if "-c" in cmd and cmd[0].endswith("g++"):
            dirs = [cmd[i + 1] for i, a in enumerate(cmd) if a == "-isystem"]
            if not any(os.path.exists(os.path.join(d, "Python.h")) for d in dirs):
                return SimpleNamespace(returncode=1, stdout="", stderr="Python.h: No such file or directory")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmoe_w4.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_expert16.so"))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "_nvcc", lambda: "/nowhere/nvcc")
    monkeypatch.setattr(B, "subprocess", SimpleNamespace(run=run))
    monkeypatch.delenv("CXX", raising=False)
    return ran


def test_a_second_build_does_nothing(tree):
    assert os.path.exists(B.build()) and os.path.exists(B.BINDING)
    n = len(tree)
    B.build()
    assert n > 2 and len(tree) == n


def test_the_binding_is_built_again_for_another_torch(tree, monkeypatch):
    """Its times say nothing of the torch and the interpreter it was compiled for."""
    B.build()
    n = len(tree)
    monkeypatch.setattr(B, "_torch_version", lambda: "/another/torch 9.9.9", raising=False)
    B.build()
    assert len(tree) > n
    n = len(tree)
    B.build()
    assert len(tree) == n
    monkeypatch.setattr(B, "sysconfig", SimpleNamespace(get_path=sysconfig.get_path, get_config_var=lambda name: "cpython-999"))
    B.build()
    assert len(tree) > n


@pytest.mark.parametrize("without", ["headers", "torch"])
def test_library_is_built_where_the_binding_cannot_be(tree, tmp_path, monkeypatch, capsys, without):
    if without == "headers":
        monkeypatch.setattr(B, "sysconfig", SimpleNamespace(get_path=lambda name: str(tmp_path)))
    else:
        find = B.importlib.util.find_spec
        monkeypatch.setattr(B.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    assert B.build() == B.LIB and os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    assert "binding" in capsys.readouterr().err
    n = len(tree)
    B.build()  # and it is up to date
    assert len(tree) == n


def test_library_is_there_when_the_binding_does_not_compile(tree, monkeypatch):
    real = B.subprocess.run

    def run(cmd, **kw):
        if "-c" in cmd and cmd[0].endswith("g++"):
            return SimpleNamespace(returncode=1, stdout="", stderr="error")
        return real(cmd, **kw)

    monkeypatch.setattr(B, "subprocess", SimpleNamespace(run=run))
    with pytest.raises(RuntimeError, match="expert16_binding"):
        B.build()
    assert os.path.exists(B.LIB)


MOVED = """
import os, sys
import bit_quantized_expert_moe_gb300 as M
M.grouped_mm
maps = {line.split()[-1] for line in open("/proc/self/maps") if line.rstrip().endswith(".so")}
print(*sorted(p for p in maps if "libmoe_w4" in p or "_expert16" in p))
"""


@pytest.mark.skipif(not os.path.exists("/proc/self/maps"), reason="needs /proc")
def test_a_moved_tree_loads_its_own_library(tmp_path):
    """The binding finds the library beside itself, not where it was linked."""
    try:
        B.build()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    pytest.importorskip("torch")
    here = tmp_path / os.path.basename(B.PKG)
    shutil.copytree(B.PKG, here, ignore=shutil.ignore_patterns("_build", "csrc", "__pycache__"))
    r = subprocess.run([sys.executable, "-c", MOVED], cwd=tmp_path, capture_output=True, text=True, check=True)
    assert r.stdout.split() == [str(here / "_expert16.so"), str(here / "libmoe_w4.so")]
