"""Building the compiled host path: optional, and only used with the Python and the
torch that it was compiled for."""
import importlib.util
import os
import subprocess
import sys
import sysconfig
import types

import pytest
import torch

from w4a4_gemm_nvfp4_b200 import _lib as L
from w4a4_gemm_nvfp4_b200 import build as B


@pytest.fixture
def elsewhere(tmp_path, tmp_path_factory, monkeypatch):
    """Outputs in folders of their own."""
    monkeypatch.setattr(B, "BUILD", str(tmp_path_factory.mktemp("objects")))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "FAST", str(tmp_path / os.path.basename(B.FAST)))
    return tmp_path


def test_left_out_without_torch(elsewhere, monkeypatch, capsys):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    B.build_fastcall()
    assert "torch" in capsys.readouterr().err and not os.path.exists(B.FAST)


def test_left_out_without_a_compiler(elsewhere, monkeypatch, capsys):
    monkeypatch.setenv("CXX", str(elsewhere / "no-such-compiler"))
    B.build_fastcall()
    assert "no-such-compiler" in capsys.readouterr().err and not os.path.exists(B.FAST)


def test_left_out_without_the_headers(elsewhere, monkeypatch, capsys):
    paths = dict(sysconfig.get_paths(), include=str(elsewhere))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    B.build_fastcall()
    assert "Python.h" in capsys.readouterr().err and not os.path.exists(B.FAST)


def test_left_out_when_it_does_not_compile(elsewhere, monkeypatch, capsys):
    def run(cmd, **kw):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(subprocess, "run", run)
    B.build_fastcall()
    assert "_fastcall" in capsys.readouterr().err and not os.path.exists(B.FAST)
    assert not os.listdir(elsewhere), "nothing half-built stays"


def test_a_module_left_out_takes_an_old_one_with_it(elsewhere, monkeypatch, capsys):
    """One that was built for something else is not left to be imported."""
    (elsewhere / "_fastcall.so").write_bytes(b"untagged, of an older build")
    with open(B.FAST, "wb") as f:
        f.write(b"of another torch")
    monkeypatch.setenv("CXX", str(elsewhere / "no-such-compiler"))
    B.build_fastcall(force=True)
    assert os.listdir(elsewhere) == []


def test_is_named_for_this_python():
    assert os.path.basename(B.FAST) == "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX")


@pytest.mark.parametrize("what", ["torch", "python", "source"])
def test_is_built_again_for_another(what, elsewhere, monkeypatch):
    """Each of what it is compiled from and for makes it stale, whatever the files'
    times say."""
    built = []

    def run(cmd, **kw):
        built.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"a module")

    monkeypatch.setattr(subprocess, "run", run)
    B.build_fastcall()
    B.build_fastcall()
    assert len(built) == 1 and os.path.exists(B.FAST)
    if what == "torch":
        monkeypatch.setattr(B, "torch_version", lambda: "0.0.1")
    elif what == "python":
        monkeypatch.setattr(sys, "version", "3.99.0 (another)")
    else:
        os.utime(B.FAST, (0, 0))
    B.build_fastcall()
    assert len(built) == 2
    B.build_fastcall()
    assert len(built) == 2


def test_one_of_another_torch_is_not_used(monkeypatch):
    used = L._fast()
    assert used and used.built_for == torch.__version__
    monkeypatch.setattr(L, "_F", None)
    other = types.ModuleType("w4a4_gemm_nvfp4_b200._fastcall")
    other.built_for = "0.0.1"
    import w4a4_gemm_nvfp4_b200 as package

    monkeypatch.setitem(sys.modules, other.__name__, other)
    monkeypatch.setattr(package, "_fastcall", other, raising=False)
    assert L._fast() is False
    monkeypatch.setattr(L, "_F", None)
    del other.built_for  # one from before it said so
    assert L._fast() is False
