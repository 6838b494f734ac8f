"""The order of the build: the C library is there whatever becomes of the Python binding."""
import importlib.util
import os
import subprocess

import pytest

from onnx_matmul_family_amd import build as b


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """No compiler runs: every object and the link's output are empty files in tmp_path."""
    ran = []

    def link(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libomm.so"))
    monkeypatch.setattr(b, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(b, "_compile", lambda src, verbose: str(tmp_path / (src + ".o")))
    monkeypatch.setattr(subprocess, "check_call", link)
    return ran


def test_library_without_torch(fake, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(b, "_build_native", lambda verbose: pytest.fail("needs torch"))
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert len(fake) == 1 and "_native.so is not built" in capsys.readouterr().err


def test_library_stays_if_the_binding_fails(fake, monkeypatch):
    def broken(verbose):
        raise RuntimeError("compile failed: binding.cpp")

    monkeypatch.setattr(b, "_build_native", broken)
    with pytest.raises(RuntimeError):
        b.build()
    assert os.path.exists(b.LIB)


def test_one_compiler_for_both(monkeypatch):
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "stopped")

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises(RuntimeError):
        b._build_native(False)
    assert ran[0][0] == b.hipcc()
